// lisa_attn_token.cu -- cross attention of a few query rows per key head (bf16):
// the single-token form, read by one pass over the keys and values.
//
// The rows that share a key head (its query heads times the queries) are the 16
// rows of a warp-level product, so every key and value is read once for all of
// them.  A cluster of CTAs shares the keys of one (batch, key head); a warp
// walks every fourth chunk of 32 keys of its CTA's part with its own ring of
// asynchronous copies, keeps the running maximum, sum and output in registers,
// and the warps and then the CTAs of the cluster join in a fixed order.  Bound
// by the bytes of K and V: no CTA waits for another until the end, and each warp
// has two chunks of 8 KB in flight (three chunks, so fewer CTAs per SM, were
// slower: 52 us against 46 at one setting of the rest).  64 x 4096 keys, 12 heads
// on 4, lengths from 0 up, from cold caches: 43 us for 137 MB, 3.2 TB/s; 256 x 4096
// keys at full length 184 us, 5.8 TB/s.
#include <algorithm>

#include "lisa_attn_tc.cuh"

namespace lisa {
namespace attn {
namespace {

constexpr int kTokenThreads = 128, kTokenWarps = 4;
constexpr int kChunk = 32;       // keys of one step
constexpr int kTokenStages = 2;

struct TokenParams {
    Problem p;
    int rows, rtiles;            // query rows per key head, tiles of 16 of them
    int splits;                  // CTAs of a cluster
    FastDiv div_rtiles, div_n;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
    const int bytes = in ? 16 : 0;   // 0: the 16 bytes are filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory of a CTA: the warps' rings, reused at the end for their results.
template <int D>
struct TokenSmem {
    static constexpr int kTileB = kChunk * D * 2;                     // K or V chunk
    static constexpr int kRing = kTokenWarps * kTokenStages * 2 * kTileB;
    static constexpr int kOut = (kTokenWarps + 1) * 16 * (D + 4) * 4;  // each warp's output and the CTA's
    static constexpr int kMain = kRing > kOut ? kRing : kOut;
};

// Byte offset of 16-byte piece c of a row of D bf16: pieces of a row permuted so
// that eight rows' pieces of one column lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t piece(int row, int c) {
    constexpr int kPieces = D / 8;
    constexpr int kRowsPer128 = 8 / kPieces;   // rows that fill the 32 banks together
    return (uint32_t)(row * D * 2) + (uint32_t)((c ^ ((row / kRowsPer128) & (kPieces - 1))) << 4);
}

template <int D, int kBias>
__global__ void __launch_bounds__(kTokenThreads) token_attention(const __grid_constant__ TokenParams x) {
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float stat_s[kTokenWarps + 1][2][16];   // maximum (in log2 units) and sum, per warp and joined
    const Problem &p = x.p;
    using S = TokenSmem<D>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
    const int split_id = blockIdx.x, b = blockIdx.z;
    int rt = blockIdx.y;
    const int kvh = split(rt, x.div_rtiles);
    float *lut = reinterpret_cast<float *>(sm + S::kMain);
    const uint32_t ring = smem_u32(sm) + (uint32_t)warp * (kTokenStages * 2 * S::kTileB);
    chain_begin();

    const int len = keys_of(p, b);
    const int chunks = (len + kChunk - 1) / kChunk, per = (chunks + x.splits - 1) / x.splits;
    const int c0 = min(split_id * per, chunks), c1 = min(c0 + per, chunks);
    const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(p.K.p) + (long long)b * p.K.sb + (long long)kvh * p.K.sh;
    const __nv_bfloat16 *V = static_cast<const __nv_bfloat16 *>(p.V.p) + (long long)b * p.V.sb + (long long)kvh * p.V.sh;
    constexpr int kPieces = D / 8, kRowsAtOnce = 32 / kPieces;
    auto load = [&](int c, int stage) {
        if (c < c1) {
            const uint32_t kd = ring + (uint32_t)(stage * 2) * S::kTileB, vd = kd + S::kTileB;
            const int r0 = lane / kPieces, pc = lane % kPieces;
#pragma unroll
            for (int e = 0; e < kChunk / kRowsAtOnce; ++e) {
                const int r = e * kRowsAtOnce + r0, j = c * kChunk + r;
                const bool in = j < len;
                copy16(kd + piece<D>(r, pc), K + (in ? (long long)j * p.K.st + 8 * pc : 0), in);
                copy16(vd + piece<D>(r, pc), V + (in ? (long long)j * p.V.st + 8 * pc : 0), in);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int s = 0; s < kTokenStages; ++s) load(c0 + warp + kTokenWarps * s, s);

    // query rows g and g + 8 of the tile: (head of the group, query)
    int row[2], head[2], qi[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        row[e] = rt * 16 + g + 8 * e;
        qi[e] = row[e];
        head[e] = kvh * p.group + split(qi[e], x.div_n);
    }
    uint32_t a[D / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const bool in = row[e] < x.rows;
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.Q.p) + (long long)b * p.Q.sb +
                                 (long long)head[e] * p.Q.sh + (long long)qi[e] * p.Q.st + 2 * q4;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            a[ks][e] = in ? *reinterpret_cast<const uint32_t *>(q + 16 * ks) : 0u;
            a[ks][2 + e] = in ? *reinterpret_cast<const uint32_t *>(q + 16 * ks + 8) : 0u;
        }
    }
    // bias: the tile's heads' values of the offsets that this CTA's keys can meet
    const float scale2 = p.scale * kLog2e;
    int lut0 = 0, lutn = 0, off[2] = {0, 0};
    if (kBias) {
        const int start = bias_start(p.bias, b), last = p.bias.entries - 1, s0 = start + p.bias.lo_c;
        // offset index of pair (i, j): step j - i - s0, clamped
        lut0 = min(max(p.bias.step_c * (c0 * kChunk) - (p.n - 1) - s0, 0), last);
        const int hi = min(max(p.bias.step_c * (min(c1 * kChunk, len) - 1) - s0, 0), last);
        lutn = max(hi - lut0 + 1, 1);
        const int h0 = kvh * p.group + quotient(rt * 16, x.div_n);
        const int h1 = kvh * p.group + quotient(min(rt * 16 + 15, x.rows - 1), x.div_n);
        const int total = (h1 - h0 + 1) * lutn;
        for (int e = tid; e < total; e += kTokenThreads) {
            const int hh = e / lutn, o = e - hh * lutn;
            lut[e] = masked_entry(__ldg(p.bias.table + (size_t)entry_bucket(p.bias, lut0 + o) * p.bias.heads + h0 + hh)) * kLog2e;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) off[e] = (min(head[e], h1) - h0) * lutn;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) qi[e] += s0 + lut0;
    }

    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    int stage = 0;
    for (int c = c0 + warp; c < c1; c += kTokenWarps) {
        copy_wait<kTokenStages - 1>();
        __syncwarp();
        const uint32_t kd = ring + (uint32_t)(stage * 2) * S::kTileB, vd = kd + S::kTileB;
        float s[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        const int mi = lane >> 3, mr = lane & 7;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4(kd + piece<D>(8 * (j + (mi >> 1)) + mr, 2 * ks + (mi & 1)), b0, b1, b2, b3);
                mma_bf16_16816(s[j], a[ks][0], a[ks][1], a[ks][2], a[ks][3], b0, b1);
                mma_bf16_16816(s[j + 1], a[ks][0], a[ks][1], a[ks][2], a[ks][3], b2, b3);
            }
        // s[j][2 e + u]: row g + 8 e, key 8 j + 2 q4 + u
        const int j0 = c * kChunk + 2 * q4;
        const bool whole = c * kChunk + kChunk <= len;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int key = j0 + 8 * j + u;
                    float v = s[j][2 * e + u] * scale2;
                    if (kBias) v += lut[off[e] + min(max(p.bias.step_c * key - qi[e], 0), lutn - 1)];
                    s[j][2 * e + u] = whole || key < len ? v : -INFINITY;
                }
        uint32_t w[4][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float t = top[e];
#pragma unroll
            for (int j = 0; j < 4; ++j) t = fmaxf(t, fmaxf(s[j][2 * e], s[j][2 * e + 1]));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
            const float ref = t == -INFINITY ? 0.f : t;   // nothing but -inf so far: weights 0, not NaN
            const float f = ex2_approx(top[e] - ref);
            top[e] = t;
            sum[e] *= f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][2 * e] *= f;
                o[j][2 * e + 1] *= f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p0 = ex2_approx(s[j][2 * e] - ref), p1 = ex2_approx(s[j][2 * e + 1] - ref);
                sum[e] += p0 + p1;
                w[j][e] = pack_bf16(p0, p1);
            }
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int j = 0; j < D / 8; j += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(vd + piece<D>(16 * kk + 8 * (mi & 1) + mr, j + (mi >> 1)), b0, b1, b2, b3);
                mma_bf16_16816(o[j], w[2 * kk][0], w[2 * kk][1], w[2 * kk + 1][0], w[2 * kk + 1][1], b0, b1);
                mma_bf16_16816(o[j + 1], w[2 * kk][0], w[2 * kk][1], w[2 * kk + 1][0], w[2 * kk + 1][1], b2, b3);
            }
        __syncwarp();   // every lane is past its reads of this stage
        load(c + kTokenWarps * kTokenStages, stage);
        stage = stage + 1 == kTokenStages ? 0 : stage + 1;
    }
    copy_wait<0>();
    __syncthreads();

    // ---- the warps' results, then the CTA's: out = sum_w 2^(top_w - top) o_w
    constexpr int kPitch = D + 4;
    float *part = reinterpret_cast<float *>(sm) + warp * 16 * kPitch;
    float *joined = reinterpret_cast<float *>(sm) + kTokenWarps * 16 * kPitch;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 2);
        if (q4 == 0) {
            stat_s[warp][0][g + 8 * e] = top[e];
            stat_s[warp][1][g + 8 * e] = sum[e];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2 *>(part + (g + 8 * e) * kPitch + 8 * j + 2 * q4) =
                make_float2(o[j][2 * e], o[j][2 * e + 1]);
    }
    __syncthreads();
    const int cl = x.splits;
    for (int e = tid; e < 16 * (D / 4); e += kTokenThreads) {
        const int r = e / (D / 4), d = 4 * (e % (D / 4));
        float t = -INFINITY, l = 0.f;
#pragma unroll
        for (int wv = 0; wv < kTokenWarps; ++wv) t = fmaxf(t, stat_s[wv][0][r]);
        const float ref = t == -INFINITY ? 0.f : t;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int wv = 0; wv < kTokenWarps; ++wv) {
            const float f = ex2_approx(stat_s[wv][0][r] - ref);
            const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(sm) + (wv * 16 + r) * kPitch + d);
            l = fmaf(f, stat_s[wv][1][r], l);
            v.x = fmaf(f, y.x, v.x);
            v.y = fmaf(f, y.y, v.y);
            v.z = fmaf(f, y.z, v.z);
            v.w = fmaf(f, y.w, v.w);
        }
        *reinterpret_cast<float4 *>(joined + r * kPitch + d) = v;
        if (d == 0) {
            stat_s[kTokenWarps][0][r] = t;
            stat_s[kTokenWarps][1][r] = l;
        }
    }
    if (cl > 1) cluster_sync();
    else __syncthreads();
    // ---- the cluster's CTAs share the rows out and add the parts up in rank order
    const uint32_t rank = cl > 1 ? cluster_rank() : 0u;
    const uint32_t joined_a = smem_u32(joined), stat_a = smem_u32(&stat_s[kTokenWarps][0][0]);
    for (int e = tid; e < 16 * (D / 4); e += kTokenThreads) {
        const int r = e / (D / 4), d = 4 * (e % (D / 4)), at = rt * 16 + r;
        if ((uint32_t)r % (uint32_t)cl != rank || at >= x.rows) continue;
        float t = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cl == 1) {
            t = stat_s[kTokenWarps][0][r];
            l = stat_s[kTokenWarps][1][r];
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
            const float ref = t == -INFINITY ? 0.f : t;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < cl) {
                    const float f = ex2_approx(tops[c] - ref);
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

template <int D, int kBias>
cudaError_t go(const TokenParams &x, cudaStream_t s) {
    cudaError_t e = allow_smem<token_attention<D, kBias>>();
    if (e != cudaSuccess) return e;
    // a tile's 16 rows belong to at most 16 heads; offsets beyond what one CTA's keys can meet are never read
    const int heads = kBias ? std::min(16, x.p.group) : 0;
    const int bytes = TokenSmem<D>::kMain + heads * x.p.bias.entries * 4;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)x.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)x.splits, (unsigned)(x.p.kv_heads * x.rtiles), (unsigned)x.p.B);
    cfg.blockDim = kTokenThreads;
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = x.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, token_attention<D, kBias>, x);
}

}  // namespace

bool token_applies(int kv_heads, int group, int n, const BiasDev &bias) {
    // Up to two row tiles per key head read the keys twice at most (the second time from L2); a sequence's offset tables
    // of the tile's heads fit beside the rings.  From cold caches, this path and tiles: 32 rows (8 heads of a group, 4
    // queries) of 256 key heads on 2048 keys 45 and 182 us, 32 rows of one head on 512 keys 21 and 20, 48 rows of one head
    // 24 and 20.  Rows of many heads would do well here beyond 32 (48 rows of 12 heads: 59 and 269).
    if ((long long)n * group > 32 || kv_heads * 2LL > 65535 || bias.mode == 2) return false;
    return bias.mode == 0 || std::min(16, group) * bias.entries <= 8192;
}

cudaError_t launch_token(const Problem &p, cudaStream_t s) {
    TokenParams x{};
    x.p = p;
    x.rows = p.n * p.group;
    x.rtiles = (x.rows + 15) / 16;
    x.div_rtiles = fast_div(x.rtiles);
    x.div_n = fast_div(p.n);
    // Two CTAs per SM at most, of 256 keys at least: a CTA's start and the join cost some microseconds, so a second
    // wave does not pay (from cold caches: 256 key heads of 4096 keys 59 us whole, 75 in two parts, 69 in four; 64 of them
    // 33 us whole, 23 in four parts, 29 in eight; 8 of 32768 keys 184 and 34 us whole and in eight).  Lengths that differ
    // even out with twice as many, while 1024 keys are left to each (256 key heads, lengths from 0 to 4096: 44 us
    // whole, 42 in two to four parts, 50 in eight; from 0 to 1000: 19 us whole, 21 in two parts, 24 in four).
    const long long ctas = (long long)p.B * p.kv_heads * x.rtiles;
    long long splits = std::min<long long>(2 * kSms / ctas, p.m / 256);
    if (p.kv_lens) splits = std::max(splits, std::min<long long>(4 * kSms / ctas, p.m / 1024));
    x.splits = (int)std::max<long long>(1, std::min<long long>(8, splits));
    if (p.d == 16) return p.bias.mode ? go<16, 1>(x, s) : go<16, 0>(x, s);
    if (p.d == 32) return p.bias.mode ? go<32, 1>(x, s) : go<32, 0>(x, s);
    return p.bias.mode ? go<64, 1>(x, s) : go<64, 0>(x, s);
}

}  // namespace attn
}  // namespace lisa
