// lisa_attn_simt.cu -- cross attention on the CUDA cores: fp32, head widths 16,
// 32 and 64, any lengths and strides.
//
// Forward, per 64 queries of one (batch, head): one pass over the keys in tiles
// of 64 with the running maximum and sum of the softmax; scores and weights
// stay in shared memory.  Backward: the dQ kernel walks the keys of 64 queries
// and also leaves delta_i = sum_j p_ij dP_ij / sum_j p_ij; the dK / dV kernel walks the
// queries (and the heads that share the keys) of 64 keys; the bias kernel
// walks the batch for one 64 x 64 tile of pairs and keeps the tile's dS sum in
// registers, so the sum over the batch has a fixed order.
//
// 256 threads as 16 x 16; thread (ty, tx) owns rows 4 ty .. 4 ty + 3 and
// columns tx + 16 c of a 64 x 64 tile, so the 16 threads of a row are one half
// of a warp and its maximum and sum are shuffles.
//
// Bound by fp32 arithmetic and shared-memory loads where there are tiles enough
// (8 entries, 8 heads of 64, 512 x 512: forward 148 us, 29 TFLOP/s, backward 510 us),
// by a tile's latency where there are few (4 entries, 2 heads of 16, 196 x 196, 32
// CTAs: 16 and 39 us), all from cold caches.
#include <algorithm>

#include <cuda_runtime.h>

#include "lisa_attn.h"
#include "lisa_bias_dev.cuh"
#include "lisa_launch.cuh"

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

__device__ __forceinline__ int valid_keys(const Problem &p, int b) {
    return p.kv_lens ? min(max(p.kv_lens[b], 0), p.m) : p.m;
}

// Scores of the tile: scale q.k + bias, -inf for keys at or behind `len`.
__device__ __forceinline__ void finish_scores(float (&s)[4][4], const Problem &p, const float *lut, int j0, int len,
                                              int tx, const int (&oq)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
        const int ok = p.bias.mode ? off_key(p.bias, j) : 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v = s[r][c] * p.scale;
            if (p.bias.mode) v += lut[min(max(ok - oq[r], 0), p.bias.entries - 1)];
            s[r][c] = j < len ? v : -INFINITY;
        }
    }
}

__device__ __forceinline__ const float *slice(const Tensor &t, int b, int h) {
    return static_cast<const float *>(t.p) + (long long)b * t.sb + (long long)h * t.sh;
}

// Shared memory: Q, K, V (dO) tiles [64][D + 4], weights [64][68], the offset table.
template <int D>
constexpr int tile_floats() { return kTile * (D + 4); }
constexpr int kWeights = kTile * (kTile + 4);

template <int D>
__global__ void __launch_bounds__(kThreads) simt_forward(const __grid_constant__ Problem p) {
    extern __shared__ __align__(16) float sm[];
    chain_begin();
    float *q_s = sm, *k_s = q_s + tile_floats<D>(), *v_s = k_s + tile_floats<D>(), *p_s = v_s + tile_floats<D>();
    float *lut = p_s + kWeights;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int i0 = blockIdx.x * kTile, h = blockIdx.y, b = blockIdx.z, kvh = h / p.group;
    const int len = valid_keys(p, b);
    if (p.bias.mode) fill_offsets<true>(p.bias, h, lut, tid, kThreads);
    load_tile<D>(slice(p.Q, b, h), p.Q.st, i0, p.n, q_s, tid);
    int oq[4];
    const int start = p.bias.mode ? bias_start(p.bias, b) : 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) oq[r] = p.bias.mode ? off_query(p.bias, min(i0 + 4 * ty + r, p.n - 1), start) : 0;
    float top[4], sum[4], acc[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        top[r] = -INFINITY;
        sum[r] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[r][c] = 0.f;
    }
    Rows<D> kr, vr;
    kr.load(slice(p.K, b, kvh), p.K.st, 0, len, tid);
    vr.load(slice(p.V, b, kvh), p.V.st, 0, len, tid);
    for (int j0 = 0; j0 < len; j0 += kTile) {
        __syncthreads();
        kr.store(k_s, tid);
        vr.store(v_s, tid);
        __syncthreads();
        kr.load(slice(p.K, b, kvh), p.K.st, j0 + kTile, len, tid);
        vr.load(slice(p.V, b, kvh), p.V.st, j0 + kTile, len, tid);
        float s[4][4];
        tile_dot<D>(q_s, k_s, ty, tx, s);
        finish_scores(s, p, lut, j0, len, tx, oq);
        float tile_top[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) tile_top[r] = fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]));
        half_max(tile_top);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float t = fmaxf(top[r], tile_top[r]);
            const float ref = t == -INFINITY ? 0.f : t;   // a row of -inf scores so far: weights 0, not NaN
            const float old = __expf(top[r] - ref);
            float share = 0.f;                            // this thread's columns; joined at the end
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float e = __expf(s[r][c] - ref);
                share += e;
                p_s[(4 * ty + r) * (kTile + 4) + tx + 16 * c] = e;
            }
            sum[r] = fmaf(sum[r], old, share);
            top[r] = t;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[r][c] *= old;
        }
        __syncwarp();   // a row's weights are written and read by one warp
        tile_mul<D>(p_s, v_s, ty, tx, acc);
    }
    float *out = const_cast<float *>(slice(p.O, b, h));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 4 * ty + r;
        sum[r] = half_sum(sum[r]);
        if (i >= p.n) continue;
        const float inv = sum[r] != 0.f ? 1.f / sum[r] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) out[(long long)i * p.O.st + tx + 16 * c] = acc[r][c] * inv;
        if (p.lse && tx == 0)
            p.lse[((size_t)b * p.heads + h) * p.n + i] = top[r] == -INFINITY ? -INFINITY : top[r] + logf(sum[r]);
    }
}

// p_ij = exp(s_ij - lse_i); rows without a valid key (lse = -inf) give 0.
__device__ __forceinline__ float row_ref(const float *lse, size_t at, bool in) {
    const float l = in ? lse[at] : INFINITY;
    return fabsf(l) > kMaxLse ? INFINITY : l;
}

template <int D>
__global__ void __launch_bounds__(kThreads) simt_dq(const __grid_constant__ Problem p) {
    extern __shared__ __align__(16) float sm[];
    chain_begin();
    float *q_s = sm, *o_s = q_s + tile_floats<D>(), *k_s = o_s + tile_floats<D>(), *v_s = k_s + tile_floats<D>();
    float *p_s = v_s + tile_floats<D>(), *lut = p_s + kWeights;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int i0 = blockIdx.x * kTile, h = blockIdx.y, b = blockIdx.z, kvh = h / p.group;
    const int len = valid_keys(p, b);
    if (i0 == 0 && h == 0 && b == 0 && tid == 0) *p.err = 0;   // these kernels have no wait that could give up
    if (p.bias.mode) fill_offsets<true>(p.bias, h, lut, tid, kThreads);
    // delta~_i = dO_i . O_i from the forward's (rounded) output
    load_tile<D>(slice(p.O, b, h), p.O.st, i0, p.n, q_s, tid);
    load_tile<D>(slice(p.dO, b, h), p.dO.st, i0, p.n, o_s, tid);
    __syncthreads();
    float delta[4], exact[4], total[4], ref[4], acc[4][D / 16];
    int oq[4];
    const size_t row0 = ((size_t)b * p.heads + h) * p.n;
    const int start = p.bias.mode ? bias_start(p.bias, b) : 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float v = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            v = fmaf(q_s[(4 * ty + r) * (D + 4) + tx + 16 * c], o_s[(4 * ty + r) * (D + 4) + tx + 16 * c], v);
        delta[r] = half_sum(v);
        exact[r] = total[r] = 0.f;
        ref[r] = row_ref(p.lse, row0 + i0 + 4 * ty + r, i0 + 4 * ty + r < p.n);
        oq[r] = p.bias.mode ? off_query(p.bias, min(i0 + 4 * ty + r, p.n - 1), start) : 0;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[r][c] = 0.f;
    }
    __syncthreads();
    load_tile<D>(slice(p.Q, b, h), p.Q.st, i0, p.n, q_s, tid);
    Rows<D> kr, vr;
    kr.load(slice(p.K, b, kvh), p.K.st, 0, len, tid);
    vr.load(slice(p.V, b, kvh), p.V.st, 0, len, tid);
    for (int j0 = 0; j0 < len; j0 += kTile) {
        __syncthreads();
        kr.store(k_s, tid);
        vr.store(v_s, tid);
        __syncthreads();
        kr.load(slice(p.K, b, kvh), p.K.st, j0 + kTile, len, tid);
        vr.load(slice(p.V, b, kvh), p.V.st, j0 + kTile, len, tid);
        float s[4][4], dp[4][4];
        tile_dot<D>(q_s, k_s, ty, tx, s);
        tile_dot<D>(o_s, v_s, ty, tx, dp);
        finish_scores(s, p, lut, j0, len, tx, oq);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float e = 0.f, t = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float w = __expf(s[r][c] - ref[r]);
                e = fmaf(w, dp[r][c], e);
                t += w;
                p_s[(4 * ty + r) * (kTile + 4) + tx + 16 * c] = w * (dp[r][c] - delta[r]);
            }
            exact[r] += e;
            total[r] += t;
        }
        __syncwarp();
        tile_mul<D>(p_s, k_s, ty, tx, acc);
    }
    float *out = static_cast<float *>(p.dQ) + row0 * D;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 4 * ty + r;
        const float e = half_sum(exact[r]), t = half_sum(total[r]);
        if (i >= p.n) continue;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) out[(size_t)i * D + tx + 16 * c] = acc[r][c] * p.scale;
        // over sum p, which takes the rounding of lse out: the dS of a row add up to 0
        if (tx == 0) p.delta[row0 + i] = t > 0.f ? e / t : e;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) simt_dkdv(const __grid_constant__ Problem p) {
    extern __shared__ __align__(16) float sm[];
    chain_begin();
    float *k_s = sm, *v_s = k_s + tile_floats<D>(), *q_s = v_s + tile_floats<D>(), *o_s = q_s + tile_floats<D>();
    float *p_s = o_s + tile_floats<D>(), *d_s = p_s + kWeights, *lut = d_s + kWeights;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int j0 = blockIdx.x * kTile, kvh = blockIdx.y, b = blockIdx.z;
    const int len = valid_keys(p, b);
    float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dk[r][c] = dv[r][c] = 0.f;
    if (j0 < len) {
        load_tile<D>(slice(p.K, b, kvh), p.K.st, j0, len, k_s, tid);
        load_tile<D>(slice(p.V, b, kvh), p.V.st, j0, len, v_s, tid);
        const int start = p.bias.mode ? bias_start(p.bias, b) : 0;
        for (int g = 0; g < p.group; ++g) {
            const int h = kvh * p.group + g;
            const size_t row0 = ((size_t)b * p.heads + h) * p.n;
            __syncthreads();
            if (p.bias.mode) fill_offsets<true>(p.bias, h, lut, tid, kThreads);
            Rows<D> qr, dr;
            qr.load(slice(p.Q, b, h), p.Q.st, 0, p.n, tid);
            dr.load(slice(p.dO, b, h), p.dO.st, 0, p.n, tid);
            for (int i0 = 0; i0 < p.n; i0 += kTile) {
                __syncthreads();
                qr.store(q_s, tid);
                dr.store(o_s, tid);
                __syncthreads();
                qr.load(slice(p.Q, b, h), p.Q.st, i0 + kTile, p.n, tid);
                dr.load(slice(p.dO, b, h), p.dO.st, i0 + kTile, p.n, tid);
                float s[4][4], dp[4][4];
                int oq[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    oq[r] = p.bias.mode ? off_query(p.bias, min(i0 + 4 * ty + r, p.n - 1), start) : 0;
                tile_dot<D>(q_s, k_s, ty, tx, s);
                tile_dot<D>(o_s, v_s, ty, tx, dp);
                finish_scores(s, p, lut, j0, len, tx, oq);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = i0 + 4 * ty + r;
                    const float ref = row_ref(p.lse, row0 + i, i < p.n);
                    const float delta = i < p.n ? p.delta[row0 + i] : 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float w = __expf(s[r][c] - ref);
                        p_s[(4 * ty + r) * (kTile + 4) + tx + 16 * c] = w;
                        d_s[(4 * ty + r) * (kTile + 4) + tx + 16 * c] = w * (dp[r][c] - delta);
                    }
                }
                __syncthreads();
                tile_mul_t<D>(p_s, o_s, ty, tx, dv);
                tile_mul_t<D>(d_s, q_s, ty, tx, dk);
            }
        }
    }
    const size_t row0 = ((size_t)b * p.kv_heads + kvh) * p.m;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int j = j0 + 4 * ty + r;
        if (j >= p.m) continue;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            static_cast<float *>(p.dK)[(row0 + j) * D + tx + 16 * c] = dk[r][c] * p.scale;
            static_cast<float *>(p.dV)[(row0 + j) * D + tx + 16 * c] = dv[r][c];
        }
    }
}

// dS summed over the batch for one 64 x 64 tile of pairs of one head.
template <int D>
__global__ void __launch_bounds__(kThreads) simt_dbias(const __grid_constant__ Problem p) {
    extern __shared__ __align__(16) float sm[];
    chain_begin();
    float *k_s = sm, *v_s = k_s + tile_floats<D>(), *q_s = v_s + tile_floats<D>(), *o_s = q_s + tile_floats<D>();
    float *lut = o_s + tile_floats<D>();
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int jtiles = (p.m + kTile - 1) / kTile;   // both in x: up to 65536 tiles of queries
    const int j0 = (int)(blockIdx.x % jtiles) * kTile, i0 = (int)(blockIdx.x / jtiles) * kTile;
    const int h = blockIdx.z, kvh = h / p.group;
    fill_offsets<true>(p.bias, h, lut, tid, kThreads);
    float acc[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = 0.f;
    const int b1 = (int)((long long)p.B * (blockIdx.y + 1) / gridDim.y);
    for (int b = (int)((long long)p.B * blockIdx.y / gridDim.y); b < b1; ++b) {   // this part of the batch
        const int len = valid_keys(p, b);
        if (j0 >= len) continue;
        const size_t row0 = ((size_t)b * p.heads + h) * p.n;
        __syncthreads();
        load_tile<D>(slice(p.K, b, kvh), p.K.st, j0, len, k_s, tid);
        load_tile<D>(slice(p.V, b, kvh), p.V.st, j0, len, v_s, tid);
        load_tile<D>(slice(p.Q, b, h), p.Q.st, i0, p.n, q_s, tid);
        load_tile<D>(slice(p.dO, b, h), p.dO.st, i0, p.n, o_s, tid);
        __syncthreads();
        float s[4][4], dp[4][4];
        int oq[4];
        const int start = bias_start(p.bias, b);
#pragma unroll
        for (int r = 0; r < 4; ++r) oq[r] = off_query(p.bias, min(i0 + 4 * ty + r, p.n - 1), start);
        tile_dot<D>(q_s, k_s, ty, tx, s);
        tile_dot<D>(o_s, v_s, ty, tx, dp);
        finish_scores(s, p, lut, j0, len, tx, oq);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = i0 + 4 * ty + r;
            const float ref = row_ref(p.lse, row0 + i, i < p.n);
            const float delta = i < p.n ? p.delta[row0 + i] : 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(__expf(s[r][c] - ref), dp[r][c] - delta, acc[r][c]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = i0 + 4 * ty + r, j = j0 + tx + 16 * c;
            if (i < p.n && j < p.m) p.dbias[(((size_t)blockIdx.y * p.heads + h) * p.n + i) * p.m + j] = acc[r][c];
        }
}

// No keys at all (either type): o = 0, lse = -inf; 16 bytes per thread.
__global__ void __launch_bounds__(kThreads) no_keys(const __grid_constant__ Problem p, int esz) {
    chain_begin();
    const int pieces = p.d * esz / 16;
    const size_t count = (size_t)p.B * p.heads * p.n * pieces;
    for (size_t e = (size_t)blockIdx.x * kThreads + threadIdx.x; e < count; e += (size_t)gridDim.x * kThreads) {
        const size_t row = e / pieces, bh = row / p.n;
        const int piece = (int)(e % pieces), i = (int)(row % p.n), h = (int)(bh % p.heads), b = (int)(bh / p.heads);
        char *o = static_cast<char *>(const_cast<void *>(p.O.p));
        o += ((long long)b * p.O.sb + (long long)h * p.O.sh + (long long)i * p.O.st) * esz + 16 * piece;
        *reinterpret_cast<uint4 *>(o) = make_uint4(0, 0, 0, 0);
        if (piece == 0 && p.lse) p.lse[row] = -INFINITY;
    }
}

template <auto kKernel>
cudaError_t run(dim3 grid, int floats, const Problem &p, cudaStream_t s) {
    const int bytes = (floats + (p.bias.mode ? p.bias.entries : 0)) * (int)sizeof(float);
    cudaError_t e = allow_smem<kKernel>();
    if (e != cudaSuccess) return e;
    return launch_plain(kKernel, grid, kThreads, (size_t)bytes, s, p);
}

template <int D>
struct Simt {
    static constexpr int t = tile_floats<D>();
    static unsigned tiles(int x) { return (unsigned)((x + kTile - 1) / kTile); }
    static cudaError_t forward(const Problem &p, cudaStream_t s) {
        return run<simt_forward<D>>(dim3(tiles(p.n), p.heads, p.B), 3 * t + kWeights, p, s);
    }
    static cudaError_t dq(const Problem &p, cudaStream_t s) {
        return run<simt_dq<D>>(dim3(tiles(p.n), p.heads, p.B), 4 * t + kWeights, p, s);
    }
    static cudaError_t dkdv(const Problem &p, cudaStream_t s) {
        return run<simt_dkdv<D>>(dim3(tiles(p.m), p.kv_heads, p.B), 4 * t + 2 * kWeights, p, s);
    }
    static cudaError_t dbias(const Problem &p, cudaStream_t s) {
        return run<simt_dbias<D>>(dim3(tiles(p.m) * tiles(p.n), p.b_splits, p.heads), 4 * t, p, s);
    }
};

}  // namespace

#define LISA_ATTN_DISPATCH(fn) \
    (p.d == 16 ? Simt<16>::fn(p, s) : p.d == 32 ? Simt<32>::fn(p, s) : Simt<64>::fn(p, s))

int simt_dbias_splits(int B, int heads, int n, int m) {
    // fewer tiles than SMs: share the batch out, a matrix for each part
    const long long tiles = (long long)heads * ((n + kTile - 1) / kTile) * ((m + kTile - 1) / kTile);
    return (int)std::max<long long>(1, std::min<long long>(kSms / tiles, B));
}

cudaError_t launch_no_keys(const Problem &p, cudaStream_t s) {
    const int esz = p.dtype == LISA_BF16 ? 2 : 4;
    const size_t count = (size_t)p.B * p.heads * p.n * (p.d * esz / 16);
    return launch_plain(no_keys, dim3((unsigned)std::min<size_t>((count + kThreads - 1) / kThreads, kSms * 8)), kThreads, 0,
                        s, p, esz);
}

cudaError_t launch_simt_forward(const Problem &p, cudaStream_t s) { return LISA_ATTN_DISPATCH(forward); }
cudaError_t launch_simt_dq(const Problem &p, cudaStream_t s) { return LISA_ATTN_DISPATCH(dq); }
cudaError_t launch_simt_dkdv(const Problem &p, cudaStream_t s) { return LISA_ATTN_DISPATCH(dkdv); }
cudaError_t launch_simt_dbias(const Problem &p, cudaStream_t s) { return LISA_ATTN_DISPATCH(dbias); }

}  // namespace attn
}  // namespace lisa
