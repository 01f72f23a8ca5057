// lisa_cache4_attn.cu -- attention of a few newest tokens over the 4-bit cache
// (bf16 queries): one pass over the held codes.
//
// The rows that share a key head (its query heads times the queries) are the 16
// rows of a warp-level product, so every code is read and unpacked once for all
// of them.  A cluster of CTAs shares the pages of one (sequence, key head); a warp
// walks every fourth page of its CTA's part with its own ring of asynchronous
// copies (a page of one key head is one block of 4.5 KB), keeps the running
// maximum, sum and output in registers, and the warps and then the CTAs of the
// cluster join in a fixed order.
//
// Scores and outputs without unpacking to values: with c the codes, sk and sv the
// scales of token j's group u of 32 elements,
//   s_j = scale sum_u sk_ju (q_u . (136 + c_ju) - 136 sum q_u)
//   o_u = sum_j (p_j sv_ju) c_ju
// The codes are bf16 operands as they come out of the words (lisa_cache4.cuh); the
// keys' offset is taken out of the accumulator's first value, the values' by an
// exact subtraction, since p sv is rounded to bf16 and 136 times that rounding would
// be the error of o.
#include <algorithm>

#include <cuda_bf16.h>

#include "lisa_attn_tc.cuh"
#include "lisa_cache4_attn.h"

namespace lisa {
namespace cache4 {
namespace {

using namespace lisa::attn;
using namespace lisa::sm100;

constexpr int kThreads = 128, kWarps = 4;
constexpr int kStages = 3;

struct Params {
    AttnProblem p;
    int rows, rtiles;            // query rows per key head, tiles of 16 of them
    int splits;                  // CTAs of a cluster
    FastDiv div_rtiles, div_n;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// One word for each group of 32 elements, side by side.
template <int G>
__device__ __forceinline__ void ld_words(uint32_t addr, uint32_t (&w)[G]) {
    if constexpr (G == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        w[0] = ld_shared(addr);
}
// Scales of two tokens side by side: s[token][group].
template <int G>
__device__ __forceinline__ void ld_scales(uint32_t addr, float (&s)[2][G]) {
    uint32_t w[G];
    ld_words<G>(addr, w);
    if constexpr (G == 2) {
        s[0][0] = bf16_lo(w[0]); s[0][1] = bf16_hi(w[0]);
        s[1][0] = bf16_lo(w[1]); s[1][1] = bf16_hi(w[1]);
    } else {
        s[0][0] = bf16_lo(w[0]); s[1][0] = bf16_hi(w[0]);
    }
}
// The pair of codes at bits 4 i of both halves of a word, as the bf16 pair 136 + code.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) { return (w >> (4 * i) & 0x000F000Fu) | 0x43004300u; }
__device__ __forceinline__ uint32_t without_offset(uint32_t pair) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(pair), "r"(0x43084308u));
    return r;
}

// d = A B + (c0, c0, c1, c1): the rows' own first values.
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%11,%11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
constexpr float kFarRef = 0x1p20f;

// kHalves: 1 where at most 8 rows share a key head (the product's upper rows are idle), else 2.
template <int D, int kHalves>
__global__ void __launch_bounds__(kThreads) attention(const __grid_constant__ Params x) {
    using B = Block<D>;
    constexpr int G = B::G;
    constexpr int kRing = kWarps * kStages * B::kBytes;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float stat_s[kWarps + 1][2][16];   // reference (in log2 units) and sum, per warp and joined
    const AttnProblem &p = x.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
    const int split_id = blockIdx.x, b = blockIdx.z;
    int rt = blockIdx.y;
    const int kvh = split(rt, x.div_rtiles);
    const uint32_t ring = smem_u32(sm) + (uint32_t)warp * (kStages * B::kBytes);
    static_assert(kRing >= (kWarps + 1) * 16 * (D + 4) * 4, "the rings hold the warps' results at the end");
    chain_begin();

    const int len = min(max(p.lens[b], 0), p.c.width * kPage);
    const int pages = (len + kPage - 1) / kPage, per = (pages + x.splits - 1) / x.splits;
    const int c0 = min(split_id * per, pages), c1 = min(c0 + per, pages);
    const int *table = p.c.table + b * p.c.table_stride;
    const uint8_t *store = p.c.store + (size_t)kvh * B::kBytes;
    const size_t page_bytes = (size_t)p.c.kv_heads * B::kBytes;
    // the warp's pages c0 + warp + 4 k; lane l holds the place of k = 32 m + l, one that is not in the cache as -1
    int places = -1, held = -1;
    auto place = [&](int k) {
        if ((k >> 5) != held) {
            held = k >> 5;
            const int at = c0 + warp + kWarps * (32 * held + lane);
            places = at < c1 ? table[at] : -1;
            if (places >= p.c.pages) places = -1;
        }
        return __shfl_sync(0xFFFFFFFFu, places, k & 31);
    };
    // bit s: the page in slot s of the ring exists
    uint32_t there = 0;
    auto load = [&](int k, int stage) {
        if (c0 + warp + kWarps * k < c1) {
            const int at = place(k);
            there = at >= 0 ? there | 1u << stage : there & ~(1u << stage);
            if (at >= 0) {
                const uint8_t *src = store + (size_t)at * page_bytes + 16 * lane;
                const uint32_t dst = ring + (uint32_t)stage * B::kBytes + 16 * lane;
#pragma unroll
                for (int e = 0; e < (B::kBytes + 511) / 512; ++e)
                    if ((e + 1) * 512 <= B::kBytes || e * 512 + 16 * lane < B::kBytes) copy16(dst + e * 512, src + e * 512);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(s, s);

    // query rows g and g + 8 of the tile: (head of the group, query), and the keys that each sees
    int row[kHalves], qi[kHalves], head[kHalves], sees[kHalves];
    uint32_t a[G][4][kHalves];   // pairs (i, i + 4) of elements 8 q4 .. 8 q4 + 7 of each group
    float minus[G][kHalves];     // -136 times the sum of the group's elements
#pragma unroll
    for (int e = 0; e < kHalves; ++e) {
        row[e] = rt * 16 + g + 8 * e;
        qi[e] = row[e];
        head[e] = kvh * p.group + split(qi[e], x.div_n);
        sees[e] = len - (p.n - 1 - qi[e]);
        const bool in = row[e] < x.rows;
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.Q.p) + (long long)b * p.Q.sb +
                                 (long long)head[e] * p.Q.sh + (long long)qi[e] * p.Q.st + 8 * q4;
#pragma unroll
        for (int u = 0; u < G; ++u) {
            const uint4 v = in ? *reinterpret_cast<const uint4 *>(q + kGroup * u) : make_uint4(0, 0, 0, 0);
            a[u][0][e] = __byte_perm(v.x, v.z, 0x5410);
            a[u][1][e] = __byte_perm(v.x, v.z, 0x7632);
            a[u][2][e] = __byte_perm(v.y, v.w, 0x5410);
            a[u][3][e] = __byte_perm(v.y, v.w, 0x7632);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += bf16_lo(a[u][i][e]) + bf16_hi(a[u][i][e]);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            minus[u][e] = -136.f * sum;
        }
    }
    const float scale2 = p.scale * kLog2e;
    float ref[kHalves], sum[kHalves], o[G][4][4];
#pragma unroll
    for (int e = 0; e < kHalves; ++e) {
        ref[e] = -INFINITY;
        sum[e] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < G; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[u][j][0] = o[u][j][1] = o[u][j][2] = o[u][j][3] = 0.f;

    // one page: its keys from `j0`; not kWhole: some are behind what a row sees
    auto page = [&](uint32_t at, int j0, auto whole) __attribute__((always_inline)) {
        constexpr bool kWhole = decltype(whole)::value;
        float s[8][2 * kHalves];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t w[G];
            ld_words<G>(at + B::key_word(8 * j + g, q4, 0), w);
            float sk[2][G];
            ld_scales<G>(at + B::off_ks + (8 * j + 2 * q4) * 2 * G, sk);
            float acc[G][4];
#pragma unroll
            for (int u = 0; u < G; ++u) {
                const uint32_t *l = a[u][0], *m = a[u][1], *n = a[u][2], *r = a[u][3];
                constexpr bool kBoth = kHalves == 2;
                mma_from(acc[u], l[0], kBoth ? l[kHalves - 1] : 0u, m[0], kBoth ? m[kHalves - 1] : 0u, code_pair(w[u], 0),
                         code_pair(w[u], 1), minus[u][0], kBoth ? minus[u][kHalves - 1] : 0.f);
                mma_bf16_16816(acc[u], n[0], kBoth ? n[kHalves - 1] : 0u, r[0], kBoth ? r[kHalves - 1] : 0u,
                               code_pair(w[u], 2), code_pair(w[u], 3));
            }
#pragma unroll
            for (int e = 0; e < kHalves; ++e)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float v = acc[0][2 * e + t] * sk[t][0];
                    if (G == 2) v = fmaf(acc[G - 1][2 * e + t], sk[t][G - 1], v);
                    if (!kWhole) v = j0 + 8 * j + 2 * q4 + t < sees[e] ? v : -INFINITY;
                    s[j][2 * e + t] = v;
                }
        }
#pragma unroll
        for (int e = 0; e < kHalves; ++e) {
            float t = s[0][2 * e];
#pragma unroll
            for (int j = 0; j < 8; ++j) t = fmaxf(t, fmaxf(s[j][2 * e], s[j][2 * e + 1]));
            t *= scale2;
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
            t = fmaxf(fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2)), ref[e]);
            const float r = t == -INFINITY ? 0.f : t;   // nothing but -inf so far: weights 0, not NaN
            const float f = ex2_approx(ref[e] - r);
            ref[e] = t;
            // The reference's rounding is common to a row's weights of this page and all others and goes out with the sum
            // while it is small (2^20: an eighth); further out the scores are rounded as the reference was.
            float mul = scale2;
            if (__any_sync(0xFFFFFFFFu, fabsf(r) > kFarRef)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[j][2 * e] *= mul;
                    s[j][2 * e + 1] *= mul;
                }
                mul = 1.f;
            }
            float part[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    s[j][2 * e + u] = ex2_approx(fmaf(s[j][2 * e + u], mul, -r));
                    part[u] += s[j][2 * e + u];
                }
            sum[e] = fmaf(sum[e], f, part[0] + part[1]);
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[u][j][2 * e] *= f;
                    o[u][j][2 * e + 1] *= f;
                }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t w[G][4] = {};   // p sv of the step's 16 tokens, as the product's left side
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 2 * k + h;
                float sv[2][G];
                ld_scales<G>(at + B::off_vs + (8 * j + 2 * q4) * 2 * G, sv);
#pragma unroll
                for (int u = 0; u < G; ++u)
#pragma unroll
                    for (int e = 0; e < kHalves; ++e) {
                        float v[2];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            v[t] = s[j][2 * e + t] * sv[t][u];
                            // behind what the row sees a scale may be anything
                            if (!kWhole && j0 + 8 * j + 2 * q4 + t >= sees[e]) v[t] = 0.f;
                        }
                        w[u][2 * h + e] = pack_bf16(v[0], v[1]);
                    }
            }
            uint32_t lo[G], hi[G];
            ld_words<G>(at + B::off_v + B::value_half(16 * k + 2 * q4, g, 0), lo);
            ld_words<G>(at + B::off_v + B::value_half(16 * k + 8 + 2 * q4, g, 0), hi);
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_bf16_16816(o[u][j], w[u][0], w[u][1], w[u][2], w[u][3], without_offset(code_pair(lo[u], j)),
                                   without_offset(code_pair(hi[u], j)));
        }
    };
    const int all_see = len - (p.n - 1);   // keys that every row of the sequence sees
    int stage = 0;
    for (int k = 0, c = c0 + warp; c < c1; ++k, c += kWarps) {
        copy_wait<kStages - 2>();
        __syncwarp();   // the page is there for every lane, and every lane is past the slot loaded next
        load(k + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
        const uint32_t at = ring + (uint32_t)stage * B::kBytes;
        if (there >> stage & 1u) {
            if ((c + 1) * kPage <= all_see)
                page(at, c * kPage, std::true_type{});
            else
                page(at, c * kPage, std::false_type{});
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copy_wait<0>();
    __syncthreads();

    // ---- the warps' results, then the CTA's: out = sum_w 2^(ref_w - ref) o_w
    constexpr int kPitch = D + 4;
    float *part = reinterpret_cast<float *>(sm) + warp * 16 * kPitch;
    float *joined = reinterpret_cast<float *>(sm) + kWarps * 16 * kPitch;
    constexpr int kRows = 8 * kHalves;
#pragma unroll
    for (int e = 0; e < kHalves; ++e) {
        sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 2);
        if (q4 == 0) {
            stat_s[warp][0][g + 8 * e] = ref[e];
            stat_s[warp][1][g + 8 * e] = sum[e];
        }
        // column 2 q4 of the products is element 8 q4 + j of the group, column 2 q4 + 1 element 8 q4 + 4 + j
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
            for (int t = 0; t < 2; ++t)
                *reinterpret_cast<float4 *>(part + (g + 8 * e) * kPitch + kGroup * u + 8 * q4 + 4 * t) =
                    make_float4(o[u][0][2 * e + t], o[u][1][2 * e + t], o[u][2][2 * e + t], o[u][3][2 * e + t]);
    }
    __syncthreads();
    const int cl = x.splits;
    for (int e = tid; e < kRows * (D / 4); e += kThreads) {
        const int r = e / (D / 4), d = 4 * (e % (D / 4));
        float t = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t = fmaxf(t, stat_s[w][0][r]);
        const float at = t == -INFINITY ? 0.f : t;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2_approx(stat_s[w][0][r] - at);
            const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(sm) + (w * 16 + r) * kPitch + d);
            l = fmaf(f, stat_s[w][1][r], l);
            v.x = fmaf(f, y.x, v.x);
            v.y = fmaf(f, y.y, v.y);
            v.z = fmaf(f, y.z, v.z);
            v.w = fmaf(f, y.w, v.w);
        }
        *reinterpret_cast<float4 *>(joined + r * kPitch + d) = v;
        if (d == 0) {
            stat_s[kWarps][0][r] = t;
            stat_s[kWarps][1][r] = l;
        }
    }
    if (cl > 1) cluster_sync();
    else __syncthreads();
    // ---- the cluster's CTAs share the rows out and add the parts up in rank order
    const uint32_t rank = cl > 1 ? cluster_rank() : 0u;
    const uint32_t joined_a = smem_u32(joined), stat_a = smem_u32(&stat_s[kWarps][0][0]);
    for (int e = tid; e < kRows * (D / 4); e += kThreads) {
        const int r = e / (D / 4), d = 4 * (e % (D / 4)), at = rt * 16 + r;
        if ((uint32_t)r % (uint32_t)cl != rank || at >= x.rows) continue;
        float t = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cl == 1) {
            t = stat_s[kWarps][0][r];
            l = stat_s[kWarps][1][r];
            v = *reinterpret_cast<const float4 *>(joined + r * kPitch + d);
        } else {
            float tops[8], sums[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < cl) {
                    const uint32_t sa = map_rank(stat_a, (uint32_t)c);
                    tops[c] = ld_dsmem(sa + (uint32_t)r * 4u);
                    sums[c] = ld_dsmem(sa + 64u + (uint32_t)r * 4u);
                    t = fmaxf(t, tops[c]);
                }
            const float base = t == -INFINITY ? 0.f : t;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < cl) {
                    const float f = ex2_approx(tops[c] - base);
                    const float4 y = ld_dsmem4(map_rank(joined_a + (uint32_t)(r * kPitch + d) * 4u, (uint32_t)c));
                    l = fmaf(f, sums[c], l);
                    v.x = fmaf(f, y.x, v.x);
                    v.y = fmaf(f, y.y, v.y);
                    v.z = fmaf(f, y.z, v.z);
                    v.w = fmaf(f, y.w, v.w);
                }
        }
        int i = at;
        const int h = kvh * p.group + split(i, x.div_n);
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint2 out;
        out.x = pack_bf16(v.x * inv, v.y * inv);
        out.y = pack_bf16(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(const_cast<void *>(p.O.p)) + (long long)b * p.O.sb +
                                   (long long)h * p.O.sh + (long long)i * p.O.st + d) = out;
        if (d == 0 && p.lse)
            p.lse[((size_t)b * p.heads + h) * p.n + i] = t == -INFINITY ? -INFINITY : kLn2 * (t + log2f(l));
    }
    if (cl > 1) cluster_sync();   // no CTA leaves while its results are being read
}

template <int D, int kHalves>
cudaError_t go(const Params &x, cudaStream_t s) {
    cudaError_t e = allow_smem<attention<D, kHalves>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)x.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)x.splits, (unsigned)(x.p.c.kv_heads * x.rtiles), (unsigned)x.p.B);
    cfg.blockDim = kThreads;
    cfg.dynamicSmemBytes = (size_t)kWarps * kStages * Block<D>::kBytes;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = x.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, attention<D, kHalves>, x);
}

}  // namespace

cudaError_t launch_attention(const AttnProblem &p, int d, cudaStream_t s) {
    Params x{};
    x.p = p;
    x.rows = p.n * p.group;
    x.rtiles = (x.rows + 15) / 16;
    x.div_rtiles = fast_div(x.rtiles);
    x.div_n = fast_div(p.n);
    // Four CTAs per SM while each has a page for every warp.
    const long long ctas = (long long)p.B * p.c.kv_heads * x.rtiles;
    x.splits = (int)std::max<long long>(1, std::min<long long>(8, std::min<long long>(4 * kSms / ctas, p.c.width / kWarps)));
    if (x.rows <= 8) return d == 64 ? go<64, 1>(x, s) : go<32, 1>(x, s);
    return d == 64 ? go<64, 2>(x, s) : go<32, 2>(x, s);
}

}  // namespace cache4
}  // namespace lisa
