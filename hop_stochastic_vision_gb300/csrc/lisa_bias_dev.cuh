// lisa_bias_dev.cuh -- device side of the bucket rule, shared by the bias
// matrix kernels and the attention kernels.
#pragma once

#include <cuda_runtime.h>

#include "lisa_attn.h"

namespace lisa {
namespace attn {
namespace {

__device__ __forceinline__ int quotient(int n, const FastDiv &f) {
    return (int)((__umulhi(f.mul, (unsigned)n) + (unsigned)n) >> f.shift);
}
// n / d, and n becomes n % d
__device__ __forceinline__ int split(int &n, const FastDiv &f) {
    const int q = quotient(n, f);
    n -= q * (int)f.d;
    return q;
}

__device__ __forceinline__ int axis_bucket(const AxisDev &ax, int x) {
    if (!ax.log_rule) return min(max(x, -ax.D), ax.D) + ax.D;
    const int a = abs(x), side = x > 0 ? ax.half : 0;
    if (a < ax.nexact) return side + a;
    int b = ax.nexact;
    for (int t = 0; t < ax.nthr; ++t) b += a >= ax.thr[t] ? 1 : 0;
    return side + b;
}

constexpr int kFar = 1 << 30;
constexpr int kFarStart = 1 << 29;

// The offsets lo .. hi that fall into bucket b (hi < lo: none; open ends at +-kFar).
__device__ __forceinline__ void bucket_range(const AxisDev &ax, int b, int &lo, int &hi) {
    if (!ax.log_rule) {
        lo = b == 0 ? -kFar : b - ax.D;
        hi = b == 2 * ax.D ? kFar : b - ax.D;
        return;
    }
    const bool pos = b >= ax.half;
    const int k = pos ? b - ax.half : b;
    int a0, a1;   // |x| range
    if (k < ax.nexact) {
        a0 = a1 = k;
    } else {
        const int t = k - ax.nexact;   // far bucket t begins at thr[t - 1] (t = 0: at nexact)
        a0 = t == 0 ? ax.nexact : ax.thr[t - 1];
        a1 = t == ax.nthr ? kFar : ax.thr[t] - 1;
    }
    if (pos) {   // x > 0
        lo = max(a0, 1);
        hi = a1;
    } else {     // x <= 0
        lo = -a1;
        hi = -a0;
    }
    if (a1 < a0) { lo = 1; hi = 0; }
}

// Row of the bucket table behind offset entry e.
__device__ __forceinline__ int entry_bucket(const BiasDev &b, int e) {
    int dr = b.lo_r, dc = b.lo_c + e;
    if (b.mode == 2) {
        const int r = quotient(e, b.div_P);
        dr = b.lo_r + r;
        dc = b.lo_c + e - r * b.P;
    }
    return axis_bucket(b.rows, dr) * b.col_buckets + axis_bucket(b.cols, dc);
}

// Entries of -2^120 and less, the types' lowest values among them, mask as -inf
// does: in units of log2(e) they would overflow to it, or not, path by path.
__device__ __forceinline__ float masked_entry(float v) { return v <= -0x1p120f ? -INFINITY : v; }

// The head's bias of every offset into shared memory, as scores (kMask) or as
// it stands; eight loads in flight per thread (one at a time took 15 us for
// 12480 offsets).
template <bool kMask>
__device__ __forceinline__ void fill_offsets(const BiasDev &b, int head, float *out, int tid, int nthreads) {
    const float *t = b.table + head;
    for (int e0 = tid; e0 < b.entries; e0 += 8 * nthreads) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = e0 + u * nthreads < b.entries ? __ldg(t + (size_t)entry_bucket(b, e0 + u * nthreads) * b.heads) : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (e0 + u * nthreads < b.entries) out[e0 + u * nthreads] = kMask ? masked_entry(v[u]) : v[u];
    }
}

// Beyond this |lse| the weights can no longer be had from fp32 scores and lse
// (their last places are 1/8 and more): such a row gives no gradient.
constexpr float kMaxLse = 0x1p20f;

// Offset index of a pair: off_key(j) - off_query(i), then clamped to the table
// (sequence) or inside it by construction (grid).
__device__ __forceinline__ int off_key(const BiasDev &b, int j) {
    if (b.mode == 1) return b.step_c * j;
    const int r = split(j, b.div_k);
    return b.step_r * b.P * r + b.step_c * j;
}
__device__ __forceinline__ int off_query(const BiasDev &b, int i, int start) {
    if (b.mode == 1) return i + start + b.lo_c;
    const int r = split(i, b.div_q);
    return b.P * r + i - b.c0;
}
__device__ __forceinline__ int bias_start(const BiasDev &b, int batch) {
    // far starts stop where every offset is in the outermost bucket already (and sums fit an int)
    return b.starts ? min(max(b.starts[batch], -kFarStart), kFarStart) : b.start;
}

}  // namespace
}  // namespace attn
}  // namespace lisa
