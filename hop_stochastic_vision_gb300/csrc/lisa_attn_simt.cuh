// lisa_attn_simt.cuh -- pieces of the attention kernels on the CUDA cores: tiles
// of 64 tokens in shared memory, products of two tiles, row maxima and sums.
//
// 256 threads as 16 x 16; thread (ty, tx) owns rows 4 ty .. 4 ty + 3 and
// columns tx + 16 c of a 64 x 64 tile.
#pragma once

#include <cuda_runtime.h>

#include "lisa_attn.h"
#include "lisa_bias_dev.cuh"

namespace lisa {
namespace attn {
namespace {

constexpr int kTile = 64;
constexpr int kThreads = 256;

__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}

// Rows t0 .. t0 + 63 of a [tokens][D] slice, first into registers (so the loads of
// the next tile run under this tile's arithmetic), then into out[64][D + 4]; rows
// at or behind `count` are zero and are not touched in memory.
template <int D>
struct Rows {
    float v[D / 16][4];
    __device__ __forceinline__ void load(const float *base, long long st, int t0, int count, int tid) {
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {
            const int e = tid + u * kThreads, r = e / (D / 4), c = 4 * (e % (D / 4));
            v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0.f;
            if (t0 + r < count) load4(base + (long long)(t0 + r) * st + c, v[u]);
        }
    }
    __device__ __forceinline__ void store(float *out, int tid) const {
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {
            const int e = tid + u * kThreads, r = e / (D / 4), c = 4 * (e % (D / 4));
            *reinterpret_cast<float4 *>(out + r * (D + 4) + c) = make_float4(v[u][0], v[u][1], v[u][2], v[u][3]);
        }
    }
};
template <int D>
__device__ __forceinline__ void load_tile(const float *base, long long st, int t0, int count, float *out, int tid) {
    Rows<D> r;
    r.load(base, st, t0, count, tid);
    r.store(out, tid);
}

// s[r][c] = sum_d A[4 ty + r][d] B[tx + 16 c][d]
template <int D>
__device__ __forceinline__ void tile_dot(const float *A, const float *B, int ty, int tx, float (&s)[4][4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[r][c] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4 *>(A + (4 * ty + r) * (D + 4) + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4 *>(B + (tx + 16 * c) * (D + 4) + d);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[r][c] = fmaf(a[r].x, b[c].x, s[r][c]);
                s[r][c] = fmaf(a[r].y, b[c].y, s[r][c]);
                s[r][c] = fmaf(a[r].z, b[c].z, s[r][c]);
                s[r][c] = fmaf(a[r].w, b[c].w, s[r][c]);
            }
    }
}

// acc[r][c] += sum_k P[4 ty + r][k] V[k][tx + 16 c]   (P rows of kTile + 4).  Here and below the tile's sum by itself and
// then one addition: N terms lose the rounding of 64 + N / 64 additions, not of N (8192 keys: o 1.9e-6 off one by one;
// 16384 queries of 4 heads that share a key: dK and dV 4.6e-6).
template <int D>
__device__ __forceinline__ void tile_mul(const float *P, const float *V, int ty, int tx, float (&acc)[4][D / 16]) {
    float sum[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) sum[r][c] = 0.f;
#pragma unroll (D == 16 ? 8 : 2)
    for (int k = 0; k < kTile; k += 4) {
        float4 p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4 *>(P + (4 * ty + r) * (kTile + 4) + k);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const float v0 = V[(k + 0) * (D + 4) + tx + 16 * c], v1 = V[(k + 1) * (D + 4) + tx + 16 * c];
            const float v2 = V[(k + 2) * (D + 4) + tx + 16 * c], v3 = V[(k + 3) * (D + 4) + tx + 16 * c];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                sum[r][c] = fmaf(p[r].x, v0, sum[r][c]);
                sum[r][c] = fmaf(p[r].y, v1, sum[r][c]);
                sum[r][c] = fmaf(p[r].z, v2, sum[r][c]);
                sum[r][c] = fmaf(p[r].w, v3, sum[r][c]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[r][c] += sum[r][c];
}

// acc[r][c] += sum_q P[q][4 ty + r] X[q][tx + 16 c]   (transposed weights)
template <int D>
__device__ __forceinline__ void tile_mul_t(const float *P, const float *X, int ty, int tx, float (&acc)[4][D / 16]) {
    float sum[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) sum[r][c] = 0.f;
#pragma unroll 4
    for (int q = 0; q < kTile; ++q) {
        const float4 p = *reinterpret_cast<const float4 *>(P + q * (kTile + 4) + 4 * ty);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const float x = X[q * (D + 4) + tx + 16 * c];
            sum[0][c] = fmaf(p.x, x, sum[0][c]);
            sum[1][c] = fmaf(p.y, x, sum[1][c]);
            sum[2][c] = fmaf(p.z, x, sum[2][c]);
            sum[3][c] = fmaf(p.w, x, sum[3][c]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[r][c] += sum[r][c];
}

// Maximum over the 16 threads of each of four rows, the rows' exchanges side by side.
__device__ __forceinline__ void half_max(float (&v)[4]) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = fmaxf(v[r], __shfl_xor_sync(0xFFFFFFFFu, v[r], o));
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Shared memory: Q, K, V (dO) tiles [64][D + 4], weights [64][68], the offset table.
template <int D>
constexpr int tile_floats() { return kTile * (D + 4); }
constexpr int kWeights = kTile * (kTile + 4);

// p_ij = exp(s_ij - lse_i); rows without a valid key (lse = -inf) give 0.
__device__ __forceinline__ float row_ref(const float *lse, size_t at, bool in) {
    const float l = in ? lse[at] : INFINITY;
    return fabsf(l) > kMaxLse ? INFINITY : l;
}

}  // namespace
}  // namespace attn
}  // namespace lisa
