// lisa_packed_simt.cu -- attention over packed prompts on the CUDA cores: 64 x 64
// tiles in shared memory (lisa_attn_simt.cuh), fp32, head widths 16, 32, 64.
//
// A CTA takes 64 queries (forward, dQ) or 64 keys (dK, dV) of one sequence and
// head and walks the tiles of the other side that its mask leaves; a tile that
// the diagonal or the sequence's end crosses is masked pair by pair.  The units
// come from the plan's lists, whole (parts are for the tensor-core kernels).
//
// Bound by a tile's latency where there are few (sequences of 196, 1, 49, 0 and 130, 2
// heads of 16: 11, 12.5 and 15.9 us for up to four tiles one behind the other), by fp32
// arithmetic and shared-memory loads where there are many.
#include <cuda_runtime.h>

#include "lisa_attn_simt.cuh"
#include "lisa_launch.cuh"
#include "lisa_packed.h"

namespace lisa {
namespace packed {
namespace {

using namespace lisa::attn;
using lisa::packed::Problem;

__device__ __forceinline__ const float *head_of(const Tensor &t, int h, int row0) {
    return static_cast<const float *>(t.p) + (long long)h * t.sh + (long long)row0 * t.st;
}

// The CTA's 64 rows of a unit; false where there are none (the unit ends, or is another part of one).
struct Rows64 {
    int row0, len, first;
    template <int kSub>
    __device__ __forceinline__ bool of(const Lists &l) {
        const Item it = l.items[blockIdx.x / kSub];
        row0 = it.row0;
        len = it.len;
        first = it.first + kTile * (blockIdx.x % kSub);
        return it.t0 == 0 && first < len;
    }
};

// Scores of a tile of queries from i0 and keys from j0 of a sequence of `len`; -inf where the mask is.
__device__ __forceinline__ void masked_scores(float (&s)[4][4], float scale, int i0, int j0, int len, bool causal, int ty, int tx) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
#pragma unroll
        for (int r = 0; r < 4; ++r) s[r][c] = j < len && !(causal && j > i0 + 4 * ty + r) ? s[r][c] * scale : -INFINITY;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) packed_forward(const __grid_constant__ Problem p) {
    extern __shared__ __align__(16) float sm[];
    chain_begin();
    float *q_s = sm, *k_s = q_s + tile_floats<D>(), *v_s = k_s + tile_floats<D>(), *p_s = v_s + tile_floats<D>();
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, h = blockIdx.y, kvh = h / p.group;
    Rows64 w;
    if (!w.of<unit_rows(kForward) / kTile>(p.lists[kForward])) return;
    const int i0 = w.first, len = w.len, end = p.causal ? min(len, i0 + kTile) : len;
    const float *K = head_of(p.K, kvh, w.row0), *V = head_of(p.V, kvh, w.row0);
    load_tile<D>(head_of(p.Q, h, w.row0), p.Q.st, i0, len, q_s, tid);
    float top[4], sum[4], acc[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        top[r] = -INFINITY;
        sum[r] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[r][c] = 0.f;
    }
    Rows<D> kr, vr;
    kr.load(K, p.K.st, 0, end, tid);
    vr.load(V, p.V.st, 0, end, tid);
    for (int j0 = 0; j0 < end; j0 += kTile) {
        __syncthreads();
        kr.store(k_s, tid);
        vr.store(v_s, tid);
        __syncthreads();
        kr.load(K, p.K.st, j0 + kTile, end, tid);
        vr.load(V, p.V.st, j0 + kTile, end, tid);
        float s[4][4];
        tile_dot<D>(q_s, k_s, ty, tx, s);
        masked_scores(s, p.scale, i0, j0, len, p.causal, ty, tx);
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
    float *out = const_cast<float *>(head_of(p.O, h, w.row0));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 4 * ty + r;
        sum[r] = half_sum(sum[r]);
        if (i >= len) continue;
        const float inv = sum[r] != 0.f ? 1.f / sum[r] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) out[(long long)i * p.O.st + tx + 16 * c] = acc[r][c] * inv;
        if (p.lse && tx == 0)
            p.lse[h * p.lse_stride + w.row0 + i] = sum[r] == 0.f ? -INFINITY : top[r] + logf(sum[r]);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) packed_dq(const __grid_constant__ Problem p) {
    extern __shared__ __align__(16) float sm[];
    chain_begin();
    float *q_s = sm, *o_s = q_s + tile_floats<D>(), *k_s = o_s + tile_floats<D>(), *v_s = k_s + tile_floats<D>();
    float *p_s = v_s + tile_floats<D>();
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, h = blockIdx.y, kvh = h / p.group;
    if (blockIdx.x == 0 && h == 0 && tid == 0) *p.err = 0;   // these kernels have no wait that could give up
    Rows64 w;
    if (!w.of<unit_rows(kDq) / kTile>(p.lists[kDq])) return;
    const int i0 = w.first, len = w.len, end = p.causal ? min(len, i0 + kTile) : len;
    const float *K = head_of(p.K, kvh, w.row0), *V = head_of(p.V, kvh, w.row0);
    // delta~_i = dO_i . O_i from the forward's (rounded) output
    load_tile<D>(head_of(p.O, h, w.row0), p.O.st, i0, len, q_s, tid);
    load_tile<D>(head_of(p.dO, h, w.row0), p.dO.st, i0, len, o_s, tid);
    __syncthreads();
    float delta[4], exact[4], total[4], ref[4], acc[4][D / 16];
    const long long at0 = h * p.lse_stride + w.row0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float v = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            v = fmaf(q_s[(4 * ty + r) * (D + 4) + tx + 16 * c], o_s[(4 * ty + r) * (D + 4) + tx + 16 * c], v);
        delta[r] = half_sum(v);
        exact[r] = total[r] = 0.f;
        ref[r] = row_ref(p.lse, at0 + i0 + 4 * ty + r, i0 + 4 * ty + r < len);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[r][c] = 0.f;
    }
    __syncthreads();
    load_tile<D>(head_of(p.Q, h, w.row0), p.Q.st, i0, len, q_s, tid);
    Rows<D> kr, vr;
    kr.load(K, p.K.st, 0, end, tid);
    vr.load(V, p.V.st, 0, end, tid);
    for (int j0 = 0; j0 < end; j0 += kTile) {
        __syncthreads();
        kr.store(k_s, tid);
        vr.store(v_s, tid);
        __syncthreads();
        kr.load(K, p.K.st, j0 + kTile, end, tid);
        vr.load(V, p.V.st, j0 + kTile, end, tid);
        float s[4][4], dp[4][4];
        tile_dot<D>(q_s, k_s, ty, tx, s);
        tile_dot<D>(o_s, v_s, ty, tx, dp);
        masked_scores(s, p.scale, i0, j0, len, p.causal, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float e = 0.f, t = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float y = __expf(s[r][c] - ref[r]);
                e = fmaf(y, dp[r][c], e);
                t += y;
                p_s[(4 * ty + r) * (kTile + 4) + tx + 16 * c] = y * (dp[r][c] - delta[r]);
            }
            exact[r] += e;
            total[r] += t;
        }
        __syncwarp();
        tile_mul<D>(p_s, k_s, ty, tx, acc);
    }
    float *out = const_cast<float *>(head_of(p.dQ, h, w.row0));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 4 * ty + r;
        const float e = half_sum(exact[r]), t = half_sum(total[r]);
        if (i >= len) continue;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) out[(long long)i * p.dQ.st + tx + 16 * c] = acc[r][c] * p.scale;
        // over sum p, which takes the rounding of lse out: the dS of a row add up to 0
        if (tx == 0) p.delta[(size_t)h * p.tokens + w.row0 + i] = t > 0.f ? e / t : e;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) packed_dkdv(const __grid_constant__ Problem p) {
    extern __shared__ __align__(16) float sm[];
    chain_begin();
    float *k_s = sm, *v_s = k_s + tile_floats<D>(), *q_s = v_s + tile_floats<D>(), *o_s = q_s + tile_floats<D>();
    float *p_s = o_s + tile_floats<D>(), *d_s = p_s + kWeights;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, kvh = blockIdx.y;
    Rows64 w;
    if (!w.of<unit_rows(kDkv) / kTile>(p.lists[kDkv])) return;
    const int j0 = w.first, len = w.len;
    float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dk[r][c] = dv[r][c] = 0.f;
    load_tile<D>(head_of(p.K, kvh, w.row0), p.K.st, j0, len, k_s, tid);
    load_tile<D>(head_of(p.V, kvh, w.row0), p.V.st, j0, len, v_s, tid);
    for (int g = 0; g < p.group; ++g) {
        const int h = kvh * p.group + g, start = p.causal ? j0 : 0;
        const float *Q = head_of(p.Q, h, w.row0), *dO = head_of(p.dO, h, w.row0);
        const long long at0 = h * p.lse_stride + w.row0;
        const float *delta_h = p.delta + (size_t)h * p.tokens + w.row0;
        Rows<D> qr, dr;
        qr.load(Q, p.Q.st, start, len, tid);
        dr.load(dO, p.dO.st, start, len, tid);
        for (int i0 = start; i0 < len; i0 += kTile) {
            __syncthreads();
            qr.store(q_s, tid);
            dr.store(o_s, tid);
            __syncthreads();
            qr.load(Q, p.Q.st, i0 + kTile, len, tid);
            dr.load(dO, p.dO.st, i0 + kTile, len, tid);
            float s[4][4], dp[4][4];
            tile_dot<D>(q_s, k_s, ty, tx, s);
            tile_dot<D>(o_s, v_s, ty, tx, dp);
            masked_scores(s, p.scale, i0, j0, len, p.causal, ty, tx);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = i0 + 4 * ty + r;
                const float ref = row_ref(p.lse, at0 + i, i < len);
                const float delta = i < len ? delta_h[i] : 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float y = __expf(s[r][c] - ref);
                    p_s[(4 * ty + r) * (kTile + 4) + tx + 16 * c] = y;
                    d_s[(4 * ty + r) * (kTile + 4) + tx + 16 * c] = y * (dp[r][c] - delta);
                }
            }
            __syncthreads();
            tile_mul_t<D>(p_s, o_s, ty, tx, dv);
            tile_mul_t<D>(d_s, q_s, ty, tx, dk);
        }
    }
    float *out_k = const_cast<float *>(head_of(p.dK, kvh, w.row0)), *out_v = const_cast<float *>(head_of(p.dV, kvh, w.row0));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int j = j0 + 4 * ty + r;
        if (j >= len) continue;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            out_k[(long long)j * p.dK.st + tx + 16 * c] = dk[r][c] * p.scale;
            out_v[(long long)j * p.dV.st + tx + 16 * c] = dv[r][c];
        }
    }
}

template <auto kKernel>
cudaError_t run(int pass, int heads, int floats, const Problem &p, cudaStream_t s) {
    cudaError_t e = allow_smem<kKernel>();
    if (e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)p.lists[pass].n_items * (unit_rows(pass) / kTile);
    return launch_plain(kKernel, dim3(blocks, (unsigned)heads), kThreads, (size_t)floats * sizeof(float), s, p);
}

template <int D>
struct Simt {
    static constexpr int t = tile_floats<D>();
    static cudaError_t forward(const Problem &p, cudaStream_t s) {
        return run<packed_forward<D>>(kForward, p.heads, 3 * t + kWeights, p, s);
    }
    static cudaError_t backward(const Problem &p, cudaStream_t s) {
        const cudaError_t e = run<packed_dq<D>>(kDq, p.heads, 4 * t + kWeights, p, s);
        return e != cudaSuccess ? e : run<packed_dkdv<D>>(kDkv, p.kv_heads, 4 * t + 2 * kWeights, p, s);
    }
};

}  // namespace

#define LISA_PACKED_DISPATCH(fn) (p.d == 16 ? Simt<16>::fn(p, s) : p.d == 32 ? Simt<32>::fn(p, s) : Simt<64>::fn(p, s))

cudaError_t launch_simt_forward(const Problem &p, cudaStream_t s) { return LISA_PACKED_DISPATCH(forward); }
cudaError_t launch_simt_backward(const Problem &p, cudaStream_t s) { return LISA_PACKED_DISPATCH(backward); }

}  // namespace packed
}  // namespace lisa
