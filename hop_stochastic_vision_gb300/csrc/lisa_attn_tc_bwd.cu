// lisa_attn_tc_bwd.cu -- the backward cross attention on the tensor cores (bf16).
//
// Three kernels of one shape, each a persistent CTA of 20 warps around 128 x 128
// tiles of pairs whose scores and dP = dO V^T are products into tensor memory:
//   dQ     128 queries against every key; dS goes back to tensor memory as bf16
//          for dQ += dS K.  Also leaves delta_i for the two others: dO . O from
//          the rounded output (an error of one rounding of O against bf16
//          results), or sum_j p dP / sum_j p in fp32 with a bias, since its gradient is fp32,
//          and where all keys are one tile
//   dK dV  128 keys against the queries of the heads that share them, the
//          tile transposed (rows are keys): dV += P^T dO, dK += dS^T Q, the
//          queries split over CTAs when there are few key tiles, the parts added
//          in order by a second kernel
//   dbias  one tile of pairs of a head, the batch one by one, the sum of the
//          unrounded dS in registers; then folded over the offsets in shared
//          memory, so dS never goes to memory
// Scores are recomputed in each (7 products for 5) so that every sum has one
// owner: no atomics, no fp32 dQ in memory, the same bits every time.
//
// Four warpgroups share a tile by columns, 32 each, a thread per row (with two of
// 64 columns the schedulers had two warps each and issued one cycle in five:
// dK, dV 88 us against 74, dQ 75 against 67 at 8 x 4096 x 4096).
// The threads take S and dP into registers as soon as both are there, so the
// next tile's products run under this tile's arithmetic.  Two barriers to wait for
// and two to arrive at per tile: a wait costs some 100 cycles even when its phase
// is long complete, and all warps pay it together.
//
// Bound by that arithmetic and its hand-overs: a tile costs about 1900 cycles in
// dQ and 2150 in dK, dV, its products 768 and 1024; the warps issue on half of the
// cycles, tensor cores 26% and 34% busy, DRAM below 8% (8 entries, 12 heads, 500
// queries on up to 1500 keys: dQ 42 us, dK, dV 52, dbias 43).
#include "lisa_attn_tc.cuh"
#include "lisa_fold.cuh"

namespace lisa {
namespace attn {
namespace {

constexpr int kMath = 512;         // threads of arithmetic: 16 warps
constexpr int kMathWarps = kMath / 32;
constexpr int kThreads = kMath + 128;   // behind them: products (two warps), loads, a helper
constexpr int kFront = kMathWarps, kLoads = kMathWarps + 1, kBack = kMathWarps + 2, kHelper = kMathWarps + 3;
constexpr int kStrip = 32;         // columns of a thread's row
constexpr int kDkvOut = kMathWarps * 2048;   // staging blocks of the math warps
constexpr int kMaxStages = 4;
constexpr uint32_t kPair = 2 * kTileBytes / 16;   // a ring stage of two tiles, in descriptor units

struct BwdParams {
    Problem p;
    MapUse uq, uk, uv, ud, uo;
    int *err;
    int first;             // this kernel clears the error word
    int qtiles, ktiles;    // tiles of 128 queries, keys
    int splits;            // dK dV: over the (head, query tile) pairs; dbias: over the batch
    int items;
    FastDiv div_qtiles, div_ktiles, div_splits, div_B, div_group;
    int stages;
    int q_slots;           // dQ: (Q, dO) pairs held, 2 unless the offset table leaves room for one
    int off_out, off_lut, off_aux;   // dynamic shared memory, behind the tiles
};

__device__ __forceinline__ int tile_keys(int len, int t) { return min(kRows, len - t * kRows); }
__device__ __forceinline__ int tile_cols(int keys) { return (keys + 15) & ~15; }

// sum p dP / sum p from the strips' (sum p dP, sum p): the division takes the
// rounding of lse out, so the dS of a row add up to 0, as they do when one far
// bucket holds all of them (16000 rows of 6 keys: dtable 9e-6 off without it).
__device__ __forceinline__ float quotient_of(float2 a, float2 b, float2 c, float2 d) {
    const float total = (a.y + b.y) + (c.y + d.y);
    return total > 0.f ? ((a.x + b.x) + (c.x + d.x)) / total : (a.x + b.x) + (c.x + d.x);
}

__device__ __forceinline__ float neg_lse2(float l) {
    return fabsf(l) > kMaxLse ? -INFINITY : -l * kLog2e;   // rows without keys among them: every weight 2^-inf = 0
}
__device__ __forceinline__ float neg_lse2(const float *lse, size_t at, bool in) { return neg_lse2(in ? lse[at] : INFINITY); }

// Weights of a strip of a row of queries, in place: s -> 2^(scale2 s + bias - lse).
// `c0`: first column of the tile, `keys`: valid columns from there (may be <= 0).
template <int kBias, int N>
__device__ __forceinline__ void row_weights(float (&s)[N], const BiasDev &b, const float *lut, const uint16_t *key_off,
                                            int j0, int keys, int oq, int oq_lo, float scale2, float nl) {
    if (kBias == 0) {
#pragma unroll
        for (int c = 0; c < N; c += 2) fma2(s[c], s[c + 1], s[c], s[c + 1], scale2, scale2, nl, nl);
    } else if (kBias == 1) {
        const int oq_hi = oq_lo + 31, last = b.entries - 1;
        const int lo = b.step_c * j0 - oq_hi, hi = b.step_c * (j0 + max(keys, 1) - 1) - oq_lo;
        if (hi <= 0 || lo >= last) {
            const float add = nl + lut[hi <= 0 ? 0 : last];
#pragma unroll
            for (int c = 0; c < N; c += 2) fma2(s[c], s[c + 1], s[c], s[c + 1], scale2, scale2, add, add);
        } else {
            int off = b.step_c * j0 - oq;
            asm volatile("" : "+r"(off));   // not hoisted out of a loop over the batch, column by column
            if (b.step_c == 1) {   // inside the padded table
                const float *l = lut + off;
#pragma unroll
                for (int c = 0; c < N; ++c) s[c] = fmaf(s[c], scale2, l[c]) + nl;
            } else {
#pragma unroll
                for (int c = 0; c < N; ++c)
                    s[c] = fmaf(s[c], scale2, lut[min(max(off + b.step_c * c, 0), last)]) + nl;
            }
        }
    } else {
        grid_bias(s, b, lut - oq, key_off, j0, scale2);   // inside the table by construction
#pragma unroll
        for (int c = 0; c < N; c += 2) add2(s[c], s[c + 1], s[c], s[c + 1], nl, nl);
    }
    if (keys < N) {
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (c >= keys) s[c] = -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = ex2_approx(s[c]);
}

// A strip.  Columns that the products did not reach hold whatever was
// there before and are not used (a load under a condition costs copies of all).
__device__ __forceinline__ void load_strip(uint32_t taddr, float (&v)[kStrip]) {
    tmem_ld32_nowait(taddr, v);
    tc_wait_ld();
}
__device__ __forceinline__ void load_strips(uint32_t ta, float (&a)[kStrip], uint32_t tb, float (&b)[kStrip]) {
    tmem_ld32_nowait(ta, a);
    tmem_ld32_nowait(tb, b);
    tc_wait_ld();
}

__device__ __forceinline__ void arrive_warp(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
}

__device__ __forceinline__ void math_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kMath) : "memory"); }

// The products' thread waits for the last use of every ring slot, so nothing
// arrives on the CTA's barriers once it has gone.
__device__ __forceinline__ void drain(uint64_t *bar, int uses, int *err) {
    if (uses > 0 && !mbar_wait(smem_u32(bar), (uses - 1) & 1)) atomicOr(err, kErrTimeoutMma);
}
__device__ __forceinline__ int uses_of(int total, int slot, int stages) {
    return total > slot ? (total - 1 - slot) / stages + 1 : 0;
}

// ------------------------------------------------------------------------ dQ
struct DqBars {
    uint64_t q_full[2], q_empty[2], kv_full[kMaxStages], kv_empty[kMaxStages];
    uint64_t full, free, ds_full, dq_done, lut_full;   // S and dP of a tile: there, in registers
};

template <int kBias>
__global__ void __launch_bounds__(kThreads, 1)
    tc_dq(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap md,
          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
          const __grid_constant__ CUtensorMap mo, const __grid_constant__ BwdParams x) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);   // stays a shared-memory pointer
    __shared__ __align__(8) DqBars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    __shared__ float2 other[3][kRows];
    __shared__ float rows_delta[kRows];
    const Problem &p = x.p;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = smem_u32(sm);
    const uint32_t qd = base, ring = base + 3 * x.q_slots * kTileBytes;   // slots of (Q, dO, O); stages of (K, V)
    float *lut = reinterpret_cast<float *>(sm + x.off_lut) + p.bias.pad;
    uint16_t *key_off = reinterpret_cast<uint16_t *>(sm + x.off_aux);
    const Guard guard{x.err, &dead};

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bar.q_full[t]), 1);
            mbar_init(smem_u32(&bar.q_empty[t]), 1 + kMathWarps);   // the products and delta
        }
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(smem_u32(&bar.kv_full[s]), 1);
            mbar_init(smem_u32(&bar.kv_empty[s]), 1);
        }
        mbar_init(smem_u32(&bar.full), 1);
        mbar_init(smem_u32(&bar.dq_done), 1);
        mbar_init(smem_u32(&bar.free), kMathWarps);
        mbar_init(smem_u32(&bar.ds_full), kMathWarps);
        mbar_init(smem_u32(&bar.lut_full), 1);
        dead = 0;
        fence_mbar_init();
    }
    if (warp == kFront) tmem_alloc(smem_u32(&tmem_slot), 512);
    if (kBias == 2)
        for (int j = tid; j < (p.m + 127) / 128 * 128; j += kThreads) key_off[j] = (uint16_t)off_key(p.bias, min(j, p.m - 1));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    chain_begin();
    if (x.first && blockIdx.x == 0 && tid == 0) *x.err = 0;
    const uint32_t tS = tmem, tP = tmem + 128, tDs = tmem + 256, tDq = tmem + 320;

    struct Item {
        int h, b, q0, len, tiles;
    };
    auto item_of = [&](int it) {
        Item w;
        w.b = split(it, x.div_qtiles);
        w.q0 = it * kRows;
        w.h = split(w.b, x.div_B);
        w.len = keys_of(p, w.b);
        w.tiles = (w.len + kRows - 1) / kRows;
        return w;
    };

    if (warp == kHelper) {
        // nothing to help with here
    } else if (warp == kLoads) {
        if (lane == 0) {
            int kt = 0, nq = 0;
            Cursor c, cq;
            for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
                const Item w = item_of(it);
                if (w.tiles == 0) continue;
                const int qs = cq.slot, g = quotient(w.h, x.div_group);
                if (nq >= x.q_slots) wait_on(smem_u32(&bar.q_empty[qs]), cq.phase ^ 1u, guard, kErrTimeoutMma);
                cq.next(x.q_slots);
                const uint32_t f = smem_u32(&bar.q_full[qs]);
                mbar_arrive_expect_tx(f, 3 * kTileBytes);
                load_rows(qd + 3 * qs * kTileBytes, &mq, x.uq, w.q0, w.h, w.b, f);
                load_rows(qd + (3 * qs + 1) * kTileBytes, &md, x.ud, w.q0, w.h, w.b, f);
                load_rows(qd + (3 * qs + 2) * kTileBytes, &mo, x.uo, w.q0, w.h, w.b, f);
                ++nq;
                for (int j = 0; j < w.tiles; ++j, ++kt, c.next(x.stages)) {
                    const uint32_t f = smem_u32(&bar.kv_full[c.slot]), at = ring + 2 * c.slot * kTileBytes;
                    if (kt >= x.stages) wait_on(smem_u32(&bar.kv_empty[c.slot]), c.phase ^ 1u, guard, kErrTimeoutMma);
                    mbar_arrive_expect_tx(f, 2 * kTileBytes);
                    load_rows(at, &mk, x.uk, j * kRows, g, w.b, f);
                    load_rows(at + kTileBytes, &mv, x.uv, j * kRows, g, w.b, f);
                }
            }
            for (int s = 0; s < x.stages; ++s) drain(&bar.kv_empty[s], uses_of(kt, s, x.stages), x.err);
            for (int t = 0; t < x.q_slots; ++t) drain(&bar.q_empty[t], uses_of(nq, t, x.q_slots), x.err);
        }
        __syncwarp();
    } else if (warp == kFront) {
        // S and dP of each tile
        int kt = 0;
        Cursor c, cq;
        const uint64_t q0 = desc_rows(qd), k0 = desc_rows(ring), v0 = desc_rows(ring + kTileBytes);
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(it);
            if (w.tiles == 0) continue;
            const int qs = cq.slot;
            wait_on(smem_u32(&bar.q_full[qs]), cq.phase, guard, kErrTimeoutLoad);
            cq.next(x.q_slots);
            const uint64_t qa = q0 + (uint32_t)qs * (3 * kTileBytes / 16), da = qa + kTileBytes / 16;
            for (int j = 0; j < w.tiles; ++j, ++kt, c.next(x.stages)) {
                const int s = c.slot, cols = tile_cols(tile_keys(w.len, j));
                wait_on(smem_u32(&bar.kv_full[s]), c.phase, guard, kErrTimeoutLoad);
                if (kt > 0) wait_on(smem_u32(&bar.free), (kt - 1) & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                if (elect_one()) {
                    mma_rows_rows(tS, qa, k0 + (uint32_t)s * kPair, cols);
                    mma_rows_rows(tP, da, v0 + (uint32_t)s * kPair, cols);
                    tc_commit(smem_u32(&bar.full));
                    if (j == w.tiles - 1) tc_commit(smem_u32(&bar.q_empty[qs]));
                }
                __syncwarp();
            }
        }
    } else if (warp == kBack) {
        // dQ += dS K.  S and dP have read the K and V tiles: dS comes of them.
        int kt = 0;
        Cursor c;
        const uint64_t kt0 = desc_tokens(ring);
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(it);
            for (int j = 0; j < w.tiles; ++j, ++kt, c.next(x.stages)) {
                wait_on(smem_u32(&bar.ds_full), kt & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                if (elect_one()) {
                    mma_weights_rows(tDq, tDs, kt0 + (uint32_t)c.slot * kPair, tile_cols(tile_keys(w.len, j)), j > 0);
                    tc_commit(smem_u32(&bar.dq_done));
                    tc_commit(smem_u32(&bar.kv_empty[c.slot]));
                }
                __syncwarp();
            }
        }
    } else {
        const int strip = warp >> 2, c0 = kStrip * strip, wt = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const float scale2 = p.scale * kLog2e;
        int kt = 0, lut_head = -1, luts = 0;
        Cursor cq;
        float lse_next = INFINITY;
        if ((int)blockIdx.x < x.items) {
            const Item w = item_of(blockIdx.x);
            if (w.q0 + wt < p.n) lse_next = p.lse[((size_t)w.b * p.heads + w.h) * p.n + w.q0 + wt];
        }
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(it);
            if (kBias && w.h != lut_head) {
                load_offsets<kMath>(p.bias, w.h, lut, &bar.lut_full, luts, tid, guard);
                lut_head = w.h;
            }
            const int i = w.q0 + wt;
            const bool in = i < p.n;
            const size_t row = ((size_t)w.b * p.heads + w.h) * p.n + i;
            const float nl = neg_lse2(lse_next);
            {   // the next item's, as it is in memory (a use would wait for it)
                const int next = it + gridDim.x;
                lse_next = INFINITY;
                if (next < x.items) {
                    const Item y = item_of(next);
                    if (y.q0 + wt < p.n) lse_next = p.lse[((size_t)y.b * p.heads + y.h) * p.n + y.q0 + wt];
                }
            }
            const bool single = w.tiles == 1;   // delta from the tile itself, below
            if (w.tiles > 0) wait_on(smem_u32(&bar.q_full[cq.slot]), cq.phase, guard, kErrTimeoutLoad);
            // dO . O of the tile's rows, 8 lanes per row
            if (w.tiles > 1) {
                const uint32_t g_s = qd + (3 * cq.slot + 1) * kTileBytes, o_s = g_s + kTileBytes;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * warp + 4 * e + (lane >> 3);
                    const uint32_t at = sw128_offset(r, lane & 7);
                    uint4 a, b;
                    ld_shared_v4(o_s + at, a.x, a.y, a.z, a.w);
                    ld_shared_v4(g_s + at, b.x, b.y, b.z, b.w);
                    float v = bf16_lo(a.x) * bf16_lo(b.x);
                    v = fmaf(bf16_hi(a.x), bf16_hi(b.x), v);
                    v = fmaf(bf16_lo(a.y), bf16_lo(b.y), v);
                    v = fmaf(bf16_hi(a.y), bf16_hi(b.y), v);
                    v = fmaf(bf16_lo(a.z), bf16_lo(b.z), v);
                    v = fmaf(bf16_hi(a.z), bf16_hi(b.z), v);
                    v = fmaf(bf16_lo(a.w), bf16_lo(b.w), v);
                    v = fmaf(bf16_hi(a.w), bf16_hi(b.w), v);
#pragma unroll
                    for (int m = 4; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
                    if ((lane & 7) == 0) rows_delta[r] = v;
                }
            }
            math_barrier();   // also: the strips of the previous item's delta have been read
            float delta = w.tiles > 1 ? rows_delta[wt] : 0.f, exact = 0.f, total = 0.f;
            int oq = 0, oq_lo = 0;
            if (kBias) {
                const int start = bias_start(p.bias, w.b);
                oq = off_query(p.bias, kBias == 2 ? min(i, p.n - 1) : i, start);
                oq_lo = off_query(p.bias, i - lane, start);
            }
            for (int j = 0; j < w.tiles; ++j, ++kt) {
                const int keys = tile_keys(w.len, j), cols = tile_cols(keys), j0 = j * kRows + c0;
                float s[kStrip], dp[kStrip];
                wait_on(smem_u32(&bar.full), kt & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                load_strips(tS + c0 + lanes, s, tP + c0 + lanes, dp);
                tc_fence_before();
                arrive_warp(&bar.free, lane);
                row_weights<kBias, kStrip>(s, p.bias, lut, key_off, j0, keys - c0, oq, oq_lo, scale2, nl);
                if (keys - c0 < kStrip) {   // dP of keys behind the last one holds whatever their values hold
#pragma unroll
                    for (int e = 0; e < kStrip; ++e)
                        if (e >= keys - c0) dp[e] = 0.f;
                }
                uint32_t ds[kStrip / 2];
                if (kBias || single) {   // delta from the unrounded weights: the bias gradient wants it, and few keys,
                                         // where dP - delta cancels most, do without the rounding of O
                    float e0 = 0.f, e1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
                    for (int e = 0; e < kStrip; e += 2) {
                        mul2(dp[e], dp[e + 1], s[e], s[e + 1], dp[e], dp[e + 1]);
                        add2(e0, e1, e0, e1, dp[e], dp[e + 1]);
                        add2(t0, t1, t0, t1, s[e], s[e + 1]);
                    }
                    exact += e0 + e1;
                    total += t0 + t1;
                    if (single) {   // the strips' shares, where the item's O is: nothing reads that now
                        float2 *share = reinterpret_cast<float2 *>(sm + (3 * cq.slot + 2) * kTileBytes) + wt;
                        share[strip * kRows] = make_float2(exact, total);
                        math_barrier();
                        delta = quotient_of(share[0], share[kRows], share[2 * kRows], share[3 * kRows]);
                    }
#pragma unroll
                    for (int e = 0; e < kStrip; e += 2) {
                        float u, v;
                        fma2(u, v, s[e], s[e + 1], -delta, -delta, dp[e], dp[e + 1]);
                        ds[e >> 1] = pack_bf16(u, v);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < kStrip; e += 2) {
                        add2(dp[e], dp[e + 1], dp[e], dp[e + 1], -delta, -delta);
                        mul2(dp[e], dp[e + 1], dp[e], dp[e + 1], s[e], s[e + 1]);
                        ds[e >> 1] = pack_bf16(dp[e], dp[e + 1]);
                    }
                }
                // the previous dS has been read
                if (kt > 0) wait_on(smem_u32(&bar.dq_done), (kt - 1) & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                tmem_st16(tDs + c0 / 2 + lanes, ds);
                if (strip == 0 && keys < cols && w.len < p.m) {
                    // S is done with the tile: what stands behind the last key may not meet dS = 0
                    zero_rows(ring + 2 * (kt % x.stages) * kTileBytes, keys, cols, wt);
                    fence_proxy_async();
                }
                tc_wait_st();
                tc_fence_before();
                arrive_warp(&bar.ds_full, lane);
            }
            if (kBias && !single) {   // the strips' shares of delta
                if (strip > 0) other[strip - 1][wt] = make_float2(exact, total);
                math_barrier();
                if (strip == 0 && in)
                    p.delta[row] = quotient_of(make_float2(exact, total), other[0][wt], other[1][wt], other[2][wt]);
            } else if (strip == 0 && in) {
                p.delta[row] = delta;
            }
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.dQ) + (row - lane) * p.d + 16 * strip;
            if (w.tiles == 0) {   // no key: no gradient
                if (in && 16 * strip < p.d) {
                    uint4 *z = reinterpret_cast<uint4 *>(out + (size_t)lane * p.d);
                    z[0] = z[1] = make_uint4(0, 0, 0, 0);
                }
                continue;
            }
            wait_on(smem_u32(&bar.dq_done), (kt - 1) & 1, guard, kErrTimeoutMma);
            tc_fence_after();
            float o[16];
            tmem_ld16_nowait(tDq + 16 * strip + lanes, o);
            tc_wait_ld();
            tc_fence_before();
            // staged where the item's O was: its last reader was delta, before every warp's dS
            store_rows_bf16<16>(qd + (3 * cq.slot + 2) * kTileBytes + (uint32_t)warp * 1024u, o, p.scale, out, p.d,
                                p.n - (i - lane), p.d - 16 * strip, lane);
            fence_proxy_async();
            arrive_warp(&bar.q_empty[cq.slot], lane);
            cq.next(x.q_slots);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kFront) tmem_dealloc(tmem, 512);
}

// --------------------------------------------------------------------- dK, dV
struct DkvBars {
    uint64_t kv_full[2], kv_empty[2], q_full[kMaxStages], q_empty[kMaxStages];
    uint64_t aux_full[kMaxStages], aux_empty[kMaxStages];
    uint64_t full, free, w_full, w_done, lut_full;   // S and dP: there, in registers; P and dS: there, read
};

// What the arithmetic needs of a tile's queries, one entry per column.
struct QueryAux {
    float nl[kRows], minus_delta[kRows];
    int oq[kRows];
};

template <int kBias>
__global__ void __launch_bounds__(kThreads, 1)
    tc_dkdv(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap md,
            const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
            const __grid_constant__ BwdParams x) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);   // stays a shared-memory pointer
    __shared__ __align__(8) DkvBars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    const Problem &p = x.p;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = smem_u32(sm);
    const uint32_t kv = base, ring = base + 2 * x.q_slots * kTileBytes;   // slots of (K, V); stages of (Q, dO)
    float *lut = reinterpret_cast<float *>(sm + x.off_lut) + p.bias.pad;
    QueryAux *aux = reinterpret_cast<QueryAux *>(sm + x.off_aux);
    const Guard guard{x.err, &dead};

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bar.kv_full[t]), 1);
            mbar_init(smem_u32(&bar.kv_empty[t]), 1);
        }
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(smem_u32(&bar.q_full[s]), 1);
            mbar_init(smem_u32(&bar.q_empty[s]), 1);
            mbar_init(smem_u32(&bar.aux_full[s]), 1);
            mbar_init(smem_u32(&bar.aux_empty[s]), kMathWarps);
        }
        mbar_init(smem_u32(&bar.full), 1);
        mbar_init(smem_u32(&bar.w_done), 1);
        mbar_init(smem_u32(&bar.free), kMathWarps);
        mbar_init(smem_u32(&bar.w_full), kMathWarps);
        mbar_init(smem_u32(&bar.lut_full), 1);
        dead = 0;
        fence_mbar_init();
    }
    if (warp == kFront) tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    chain_begin();
    const uint32_t tS = tmem, tD = tmem + 128, tPw = tmem + 256, tDs = tmem + 320, tDv = tmem + 384, tDk = tmem + 448;
    const int steps = p.group * x.qtiles;   // (head, query tile) pairs of a kv head
    const int tail = tile_cols(p.n - (x.qtiles - 1) * kRows);   // columns of a head's last tile of queries

    struct Item {
        int g, b, j0, split, len, u0, u1;
    };
    auto item_of = [&](int it) {
        Item w;
        int jt = split(it, x.div_splits);
        w.split = it;
        w.b = split(jt, x.div_ktiles);
        w.j0 = jt * kRows;
        w.g = split(w.b, x.div_B);
        w.len = keys_of(p, w.b);
        const int per = quotient(steps + x.splits - 1, x.div_splits);
        w.u0 = min(w.split * per, steps);
        w.u1 = w.j0 < w.len ? min(w.u0 + per, steps) : w.u0;
        return w;
    };

    if (warp == kHelper) {
        // per-query scalars of each tile
        int n = 0;
        Cursor c;
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(it);
            const int start = kBias ? bias_start(p.bias, w.b) : 0;
            for (int u = w.u0; u < w.u1; ++u, ++n, c.next(x.stages)) {
                const int s = c.slot;
                if (n >= x.stages) wait_on(smem_u32(&bar.aux_empty[s]), c.phase ^ 1u, guard, kErrTimeoutMma);
                int qt = u;
                const int h = w.g * p.group + split(qt, x.div_qtiles), q0 = qt * kRows;
                const size_t row0 = ((size_t)w.b * p.heads + h) * p.n;
#pragma unroll
                for (int e = lane; e < kRows; e += 32) {
                    const int i = q0 + e;
                    const bool in = i < p.n;
                    aux[s].nl[e] = neg_lse2(p.lse, row0 + i, in);
                    aux[s].minus_delta[e] = in ? -p.delta[row0 + i] : 0.f;
                    // behind the last query: an offset whose three neighbours below are in the table too
                    if (kBias) aux[s].oq[e] = off_query(p.bias, kBias == 2 ? min(i, p.n - 1) : i, start) - (kBias == 2 && !in ? 3 : 0);
                }
                arrive_warp(&bar.aux_full[s], lane);
            }
        }
    } else if (warp == kLoads) {
        if (lane == 0) {
            int n = 0, items = 0;
            Cursor c, ck;
            for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
                const Item w = item_of(it);
                if (w.u0 >= w.u1) continue;
                if (items >= x.q_slots) wait_on(smem_u32(&bar.kv_empty[ck.slot]), ck.phase ^ 1u, guard, kErrTimeoutMma);
                ++items;
                const uint32_t f = smem_u32(&bar.kv_full[ck.slot]), kv_at = kv + 2 * ck.slot * kTileBytes;
                ck.next(x.q_slots);
                mbar_arrive_expect_tx(f, 2 * kTileBytes);
                load_rows(kv_at, &mk, x.uk, w.j0, w.g, w.b, f);
                load_rows(kv_at + kTileBytes, &mv, x.uv, w.j0, w.g, w.b, f);
                for (int u = w.u0; u < w.u1; ++u, ++n, c.next(x.stages)) {
                    const int s = c.slot;
                    const uint32_t ph = c.phase;
                    int qt = u;
                    const int h = w.g * p.group + split(qt, x.div_qtiles), q0 = qt * kRows;
                    const uint32_t f = smem_u32(&bar.q_full[s]), at = ring + 2 * s * kTileBytes;
                    if (n >= x.stages) wait_on(smem_u32(&bar.q_empty[s]), ph ^ 1u, guard, kErrTimeoutMma);
                    mbar_arrive_expect_tx(f, 2 * kTileBytes);
                    load_rows(at, &mq, x.uq, q0, h, w.b, f);
                    load_rows(at + kTileBytes, &md, x.ud, q0, h, w.b, f);
                }
            }
            for (int s = 0; s < x.stages; ++s) {
                drain(&bar.q_empty[s], uses_of(n, s, x.stages), x.err);
            }
            for (int t = 0; t < x.q_slots; ++t) drain(&bar.kv_empty[t], uses_of(items, t, x.q_slots), x.err);
        }
        __syncwarp();
    } else if (warp == kFront) {
        // S^T and dP^T of each tile
        int n = 0;
        Cursor c, ck;
        const uint64_t k0 = desc_rows(kv), v0 = desc_rows(kv + kTileBytes), q0 = desc_rows(ring),
                       d0 = desc_rows(ring + kTileBytes);
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(it);
            if (w.u0 >= w.u1) continue;
            const int ks = ck.slot;
            wait_on(smem_u32(&bar.kv_full[ks]), ck.phase, guard, kErrTimeoutLoad);
            ck.next(x.q_slots);
            const uint64_t ka = k0 + (uint32_t)ks * kPair, va = v0 + (uint32_t)ks * kPair;
            int qt = w.u0;
            split(qt, x.div_qtiles);
            for (int u = w.u0; u < w.u1; ++u, ++n, c.next(x.stages)) {
                const int s = c.slot, cols = qt == x.qtiles - 1 ? tail : kRows;
                qt = qt == x.qtiles - 1 ? 0 : qt + 1;
                wait_on(smem_u32(&bar.q_full[s]), c.phase, guard, kErrTimeoutLoad);
                if (n > 0) wait_on(smem_u32(&bar.free), (n - 1) & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                if (elect_one()) {
                    mma_rows_rows(tS, ka, q0 + (uint32_t)s * kPair, cols);
                    mma_rows_rows(tD, va, d0 + (uint32_t)s * kPair, cols);
                    tc_commit(smem_u32(&bar.full));
                    if (u == w.u1 - 1) tc_commit(smem_u32(&bar.kv_empty[ks]));
                }
                __syncwarp();
            }
        }
    } else if (warp == kBack) {
        // dV += P^T dO, dK += dS^T Q.  S^T and dP^T have read the tiles too: P and dS come of them.
        int n = 0;
        Cursor c;
        const uint64_t qt0 = desc_tokens(ring), dt0 = desc_tokens(ring + kTileBytes);
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(it);
            int qt = w.u0;
            split(qt, x.div_qtiles);
            for (int u = w.u0; u < w.u1; ++u, ++n, c.next(x.stages)) {
                const int s = c.slot, cols = qt == x.qtiles - 1 ? tail : kRows;
                qt = qt == x.qtiles - 1 ? 0 : qt + 1;
                wait_on(smem_u32(&bar.w_full), n & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                if (elect_one()) {
                    mma_weights_rows(tDv, tPw, dt0 + (uint32_t)s * kPair, cols, u > w.u0);
                    mma_weights_rows(tDk, tDs, qt0 + (uint32_t)s * kPair, cols, u > w.u0);
                    tc_commit(smem_u32(&bar.w_done));
                    tc_commit(smem_u32(&bar.q_empty[s]));
                }
                __syncwarp();
            }
        }
    } else {
        const int strip = warp >> 2, c0 = kStrip * strip, wt = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const float scale2 = p.scale * kLog2e;
        int n = 0, lut_head = -1, luts = 0;
        Cursor ca;
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(it);
            const int j = w.j0 + wt;
            const int ok = kBias ? off_key(p.bias, min(j, p.m - 1)) : 0;
            int qt = w.u0;
            int h = w.g * p.group + split(qt, x.div_qtiles);
            for (int u = w.u0; u < w.u1; ++u, ++n, ca.next(x.stages), h += qt == x.qtiles - 1, qt = qt == x.qtiles - 1 ? 0 : qt + 1) {
                if (kBias && h != lut_head) {
                    load_offsets<kMath>(p.bias, h, lut, &bar.lut_full, luts, tid, guard);
                    lut_head = h;
                }
                const int cols = tile_cols(min(kRows, p.n - qt * kRows));
                const QueryAux &a = aux[ca.slot];
                float s[kStrip], dp[kStrip];
                wait_on(smem_u32(&bar.aux_full[ca.slot]), ca.phase, guard, kErrTimeoutLoad);
                wait_on(smem_u32(&bar.full), n & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                load_strips(tS + c0 + lanes, s, tD + c0 + lanes, dp);
                tc_fence_before();
                arrive_warp(&bar.free, lane);
                if (kBias == 1) {
                    const int last = p.bias.entries - 1;
                    const int off = ok - a.oq[c0];   // column c: off - c
                    const int off_lo = __shfl_sync(0xFFFFFFFFu, off, 0), off_hi = __shfl_sync(0xFFFFFFFFu, off, 31);
                    // rows of one warp are 32 keys in order, all offsets of the strip in off_lo - 31 .. off_hi
                    if (off_hi <= 0 || off_lo - (kStrip - 1) >= last) {
                        const float add = lut[off_hi <= 0 ? 0 : last];
#pragma unroll
                        for (int c = 0; c < kStrip; c += 4) {
                            const float4 l = *reinterpret_cast<const float4 *>(a.nl + c0 + c);
                            fma2(s[c], s[c + 1], s[c], s[c + 1], scale2, scale2, l.x, l.y);
                            fma2(s[c + 2], s[c + 3], s[c + 2], s[c + 3], scale2, scale2, l.z, l.w);
                            add2(s[c], s[c + 1], s[c], s[c + 1], add, add);
                            add2(s[c + 2], s[c + 3], s[c + 2], s[c + 3], add, add);
                        }
                    } else if (p.bias.step_c == 1) {   // inside the padded table
                        const float *l = lut + off;
#pragma unroll
                        for (int c = 0; c < kStrip; ++c) s[c] = fmaf(s[c], scale2, l[-c]) + a.nl[c0 + c];
                    } else {
#pragma unroll
                        for (int c = 0; c < kStrip; ++c)
                            s[c] = fmaf(s[c], scale2, lut[min(max(off - c, 0), last)]) + a.nl[c0 + c];
                    }
                } else if (kBias == 2) {
                    const float *l4 = lut + ok;   // inside the table by construction
#pragma unroll
                    for (int c = 0; c < kStrip; c += 4) {
                        const float4 l = *reinterpret_cast<const float4 *>(a.nl + c0 + c);
                        float v[4];
                        if (p.bias.run_q) {   // four queries of one row: consecutive offsets, downwards
                            const float *at = l4 - a.oq[c0 + c];
#pragma unroll
                            for (int u = 0; u < 4; ++u) v[u] = at[-u];
                        } else {
                            const int4 o = *reinterpret_cast<const int4 *>(a.oq + c0 + c);
                            v[0] = l4[-o.x];
                            v[1] = l4[-o.y];
                            v[2] = l4[-o.z];
                            v[3] = l4[-o.w];
                        }
                        fma2(s[c], s[c + 1], s[c], s[c + 1], scale2, scale2, v[0], v[1]);
                        fma2(s[c + 2], s[c + 3], s[c + 2], s[c + 3], scale2, scale2, v[2], v[3]);
                        add2(s[c], s[c + 1], s[c], s[c + 1], l.x, l.y);
                        add2(s[c + 2], s[c + 3], s[c + 2], s[c + 3], l.z, l.w);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kStrip; c += 4) {
                        const float4 l = *reinterpret_cast<const float4 *>(a.nl + c0 + c);
                        fma2(s[c], s[c + 1], s[c], s[c + 1], scale2, scale2, l.x, l.y);
                        fma2(s[c + 2], s[c + 3], s[c + 2], s[c + 3], scale2, scale2, l.z, l.w);
                    }
                }
                uint32_t pw[kStrip / 2], ds[kStrip / 2];
#pragma unroll
                for (int e = 0; e < kStrip; e += 4) {
                    const float4 d = *reinterpret_cast<const float4 *>(a.minus_delta + c0 + e);
#pragma unroll
                    for (int u = 0; u < 4; ++u) s[e + u] = ex2_approx(s[e + u]);
                    pw[e >> 1] = pack_bf16(s[e], s[e + 1]);
                    pw[(e >> 1) + 1] = pack_bf16(s[e + 2], s[e + 3]);
                    add2(dp[e], dp[e + 1], dp[e], dp[e + 1], d.x, d.y);
                    add2(dp[e + 2], dp[e + 3], dp[e + 2], dp[e + 3], d.z, d.w);
                    mul2(dp[e], dp[e + 1], dp[e], dp[e + 1], s[e], s[e + 1]);
                    mul2(dp[e + 2], dp[e + 3], dp[e + 2], dp[e + 3], s[e + 2], s[e + 3]);
                    ds[e >> 1] = pack_bf16(dp[e], dp[e + 1]);
                    ds[(e >> 1) + 1] = pack_bf16(dp[e + 2], dp[e + 3]);
                }
                // the previous P and dS have been read
                if (n > 0) wait_on(smem_u32(&bar.w_done), (n - 1) & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                tmem_st16(tPw + c0 / 2 + lanes, pw);
                tmem_st16(tDs + c0 / 2 + lanes, ds);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&bar.aux_empty[ca.slot]));
                    mbar_arrive(smem_u32(&bar.w_full));
                }
            }
            // ---- strips 0, 1 store dV, 2 and 3 dK, 32 columns each; rows behind the last key are 0
            float o[kStrip];
            const int dk = strip >> 1, oc = kStrip * (strip & 1);
            const bool some = w.u0 < w.u1 && j < w.len;
            if (w.u0 < w.u1) wait_on(smem_u32(&bar.w_done), (n - 1) & 1, guard, kErrTimeoutMma);
            tc_fence_after();
            load_strip((dk ? tDk : tDv) + oc + lanes, o);
            tc_fence_before();
#pragma unroll
            for (int c = 0; c < kStrip; ++c) o[c] = some ? o[c] : 0.f;
            const size_t row = ((size_t)w.b * p.kv_heads + w.g) * p.m + j;
            if (x.splits == 1) {
                const int r0 = j - lane;
                store_rows_bf16<kStrip>(base + x.off_out + (uint32_t)warp * 2048u, o, dk ? p.scale : 1.f,
                                        static_cast<__nv_bfloat16 *>(dk ? p.dK : p.dV) + (row - lane) * p.d + oc, p.d,
                                        p.m - r0, p.d - oc, lane);
            } else if (j < p.m) {
                float4 *out = reinterpret_cast<float4 *>(
                    (dk ? p.dk_part : p.dv_part) + ((size_t)w.split * ((size_t)p.B * p.kv_heads * p.m) + row) * p.d + oc);
#pragma unroll
                for (int c = 0; c < kStrip; c += 4)
                    if (oc + c < p.d) out[c / 4] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kFront) tmem_dealloc(tmem, 512);
}

// dK, dV from the parts of the queries, in order.
__global__ void __launch_bounds__(256) join_dkdv(const __grid_constant__ Problem p) {
    chain_begin();
    const size_t total = (size_t)p.B * p.kv_heads * p.m * p.d;
    const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= total) return;
    const float *part = blockIdx.y ? p.dk_part : p.dv_part;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < p.q_splits; ++s) {
        const float4 a = *reinterpret_cast<const float4 *>(part + s * total + at);
        v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
    }
    const float mul = blockIdx.y ? p.scale : 1.f;
    uint2 o;
    o.x = pack_bf16(v.x * mul, v.y * mul);
    o.y = pack_bf16(v.z * mul, v.w * mul);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(blockIdx.y ? p.dK : p.dV) + at) = o;
}

// --------------------------------------------------------------------- dbias
struct DbBars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t s_full, s_free, lut_full;   // S and dP: there, in registers
};

template <int kBias>
__global__ void __launch_bounds__(kThreads, 1)
    tc_dbias(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap md,
             const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
             const __grid_constant__ BwdParams x) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);   // stays a shared-memory pointer
    __shared__ __align__(8) DbBars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    const Problem &p = x.p;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const uint32_t ring = smem_u32(sm);   // stages of (Q, dO, K, V)
    float *lut = reinterpret_cast<float *>(sm + x.off_lut) + p.bias.pad;
    uint16_t *key_off = reinterpret_cast<uint16_t *>(sm + x.off_aux);   // of the item's 128 keys
    float *tile = reinterpret_cast<float *>(sm + x.off_out), *sums = tile + kFoldTile * kFoldPitch;
    const Guard guard{x.err, &dead};

    if (tid == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(smem_u32(&bar.full[s]), 1);
            mbar_init(smem_u32(&bar.empty[s]), 1);
        }
        mbar_init(smem_u32(&bar.s_full), 1);
        mbar_init(smem_u32(&bar.s_free), kMathWarps);
        mbar_init(smem_u32(&bar.lut_full), 1);
        dead = 0;
        fence_mbar_init();
    }
    if (warp == kFront) tmem_alloc(smem_u32(&tmem_slot), 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    chain_begin();
    const uint32_t tS = tmem, tD = tmem + 128;

    struct Item {
        int h, q0, j0, split, b0, b1;
    };
    auto item_of = [&](int it) {
        Item w;
        int jt = split(it, x.div_splits);
        w.split = it;
        int qt = split(jt, x.div_ktiles);
        w.j0 = jt * kRows;
        w.h = split(qt, x.div_qtiles);
        w.q0 = qt * kRows;
        const int per = quotient(p.B + x.splits - 1, x.div_splits);
        w.b0 = min(w.split * per, p.B);
        w.b1 = min(w.b0 + per, p.B);
        return w;
    };

    if (warp >= kBack) {
        // nothing to do here
    } else if (warp == kLoads) {
        if (lane == 0) {
            int n = 0;
            Cursor c;
            for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
                const Item w = item_of(it);
                for (int b = w.b0; b < w.b1; ++b) {
                    if (w.j0 >= keys_of(p, b)) continue;
                    const int s = c.slot;
                    if (n >= x.stages) wait_on(smem_u32(&bar.empty[s]), c.phase ^ 1u, guard, kErrTimeoutMma);
                    const uint32_t f = smem_u32(&bar.full[s]), at = ring + 4 * s * kTileBytes;
                    mbar_arrive_expect_tx(f, 4 * kTileBytes);
                    load_rows(at, &mq, x.uq, w.q0, w.h, b, f);
                    load_rows(at + 2 * kTileBytes, &mk, x.uk, w.j0, quotient(w.h, x.div_group), b, f);
                    load_rows(at + kTileBytes, &md, x.ud, w.q0, w.h, b, f);
                    load_rows(at + 3 * kTileBytes, &mv, x.uv, w.j0, quotient(w.h, x.div_group), b, f);
                    ++n;
                    c.next(x.stages);
                }
            }
            for (int s = 0; s < x.stages; ++s) drain(&bar.empty[s], uses_of(n, s, x.stages), x.err);
        }
        __syncwarp();
    } else if (warp == kFront) {
        {
            int n = 0;
            Cursor c;
            const uint64_t r0 = desc_rows(ring);
            for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
                const Item w = item_of(it);
                for (int b = w.b0; b < w.b1; ++b) {
                    const int len = keys_of(p, b);
                    if (w.j0 >= len) continue;
                    const int s = c.slot, cols = tile_cols(min(kRows, len - w.j0));
                    const uint64_t at = r0 + (uint32_t)s * (4 * kTileBytes / 16);
                    wait_on(smem_u32(&bar.full[s]), c.phase, guard, kErrTimeoutLoad);
                    if (n > 0) wait_on(smem_u32(&bar.s_free), (n - 1) & 1, guard, kErrTimeoutMma);
                    tc_fence_after();
                    if (elect_one()) {
                        mma_rows_rows(tS, at, at + 2 * kTileBytes / 16, cols);
                        mma_rows_rows(tD, at + kTileBytes / 16, at + 3 * kTileBytes / 16, cols);
                        tc_commit(smem_u32(&bar.s_full));
                        tc_commit(smem_u32(&bar.empty[s]));
                    }
                    __syncwarp();
                    ++n;
                    c.next(x.stages);
                }
            }
        }
        __syncwarp();
    } else {
        const int strip = warp >> 2, c0 = kStrip * strip, wt = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const float scale2 = p.scale * kLog2e;
        int n = 0, lut_head = -1, luts = 0;
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(it);
            if (w.h != lut_head) {
                load_offsets<kMath>(p.bias, w.h, lut, &bar.lut_full, luts, tid, guard);
                lut_head = w.h;
            }
            // lse and delta of the row, one batch entry ahead, as they are in memory (a use would wait for them)
            const int i = w.q0 + wt, j0 = w.j0 + c0;
            const bool in = i < p.n;
            float lse_next = INFINITY, delta_next = 0.f;
            auto scalars = [&](int b) __attribute__((always_inline)) {
                const size_t row = ((size_t)b * p.heads + w.h) * p.n + i;
                lse_next = in && b < w.b1 ? p.lse[row] : INFINITY;
                delta_next = in && b < w.b1 ? p.delta[row] : 0.f;
            };
            scalars(w.b0);
            if (kBias == 2) {   // the previous item's are read: every warp has passed its fold
                if (tid < kRows) key_off[tid] = (uint16_t)off_key(p.bias, min(w.j0 + tid, p.m - 1));
                math_barrier();
            }
            const int oq = off_query(p.bias, kBias == 2 ? min(i, p.n - 1) : i, p.bias.start);
            const int oq_lo = off_query(p.bias, i - lane, p.bias.start);
            float acc[kStrip];
#pragma unroll
            for (int c = 0; c < kStrip; ++c) acc[c] = 0.f;
            for (int b = w.b0; b < w.b1; ++b) {
                const float nl = neg_lse2(lse_next), delta = delta_next;
                scalars(b + 1);
                const int len = keys_of(p, b);
                if (w.j0 >= len) continue;
                const int keys = min(kStrip, len - j0);
                wait_on(smem_u32(&bar.s_full), n & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                // sixteen columns at a time: with the sums of all 32 a whole strip of S and dP would not stay in
                // registers, and a spill goes to L2 (shared memory leaves next to no L1)
#pragma unroll
                for (int c = 0; c < kStrip; c += 16) {
                    float s[16], dp[16];
                    tmem_ld16_nowait(tS + c0 + c + lanes, s);
                    tmem_ld16_nowait(tD + c0 + c + lanes, dp);
                    tc_wait_ld();
                    if (c + 16 == kStrip) {
                        tc_fence_before();
                        arrive_warp(&bar.s_free, lane);
                    }
                    row_weights<kBias, 16>(s, p.bias, lut, key_off - w.j0, j0 + c, keys - c, oq, oq_lo, scale2, nl);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        add2(dp[e], dp[e + 1], dp[e], dp[e + 1], -delta, -delta);
                        if (c + e >= keys) dp[e] = 0.f;
                        if (c + e + 1 >= keys) dp[e + 1] = 0.f;
                        fma2(acc[c + e], acc[c + e + 1], s[e], s[e + 1], dp[e], dp[e + 1], acc[c + e], acc[c + e + 1]);
                    }
                }
                ++n;
            }
            float *mine = tile + wt * kFoldPitch + c0;
#pragma unroll
            for (int c = 0; c < kStrip; ++c) mine[c] = acc[c];
            math_barrier();
            if (p.folded) {
                const TileGeom g = fold_geom(p.fold, w.q0 / kFoldTile, w.j0 / kFoldTile);
                float *out = fold_block(p.fold, w.split, w.h, w.q0 / kFoldTile, w.j0 / kFoldTile);
                const bool direct = fold_direct(p.fold, g);
                fold_offsets(p.fold, g, tile, direct ? out : sums, direct ? p.fold.K : g.dc_n, tid, kMath);
                math_barrier();
                if (!direct) fold_buckets(p.fold, g, sums, out, tid, kMath);
            } else {
                float *out = p.dbias + ((size_t)w.split * p.heads + w.h) * ((size_t)p.n * p.m) + (size_t)w.q0 * p.m + w.j0;
                for (int r = warp; r < min(kRows, p.n - w.q0); r += kMathWarps)
                    for (int c = lane; c < min(kRows, p.m - w.j0); c += 32)
                        out[(size_t)r * p.m + c] = tile[r * kFoldPitch + c];
                math_barrier();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kFront) tmem_dealloc(tmem, 256);
}

struct Maps {
    CUtensorMap q, d, k, v, o;
};
bool fill_maps(Maps &m, BwdParams &x, const Problem &p) {
    x.p = p;
    x.qtiles = (p.n + kRows - 1) / kRows;
    x.ktiles = (p.m + kRows - 1) / kRows;
    x.splits = 1;
    x.div_qtiles = fast_div(x.qtiles);
    x.div_ktiles = fast_div(x.ktiles);
    x.div_splits = fast_div(1);
    x.div_B = fast_div(p.B);
    x.div_group = fast_div(p.group);
    return make_map(&m.q, &x.uq, p.Q, p.B, p.heads, p.n, p.d) && make_map(&m.d, &x.ud, p.dO, p.B, p.heads, p.n, p.d) &&
           make_map(&m.k, &x.uk, p.K, p.B, p.kv_heads, p.m, p.d) &&
           make_map(&m.v, &x.uv, p.V, p.B, p.kv_heads, p.m, p.d) && make_map(&m.o, &x.uo, p.O, p.B, p.heads, p.n, p.d);
}

template <auto kKernel>
cudaError_t go_dq(const Maps &m, const BwdParams &x, int bytes, cudaStream_t s) {
    cudaError_t e = allow_smem<kKernel>();
    if (e != cudaSuccess) return e;
    return launch_plain(kKernel, dim3((unsigned)std::min(x.items, sms())), kThreads, bytes, s, m.q, m.d, m.k, m.v, m.o, x);
}

template <auto kKernel>
cudaError_t go(const Maps &m, const BwdParams &x, int bytes, cudaStream_t s) {
    cudaError_t e = allow_smem<kKernel>();
    if (e != cudaSuccess) return e;
    return launch_plain(kKernel, dim3((unsigned)std::min(x.items, sms())), kThreads, bytes, s, m.q, m.d, m.k, m.v, x);
}

}  // namespace

int tc_dkdv_splits(int B, int kv_heads, int group, int n, int m) {
    const long long items = (long long)B * kv_heads * ((m + kRows - 1) / kRows);
    const long long steps = (long long)group * ((n + kRows - 1) / kRows);
    // At most half as many items as SMs: share the queries out in one round, at least two tiles to each part.  The
    // backward from cold caches, whole and as here: 2 items of 32 tiles 41 and 25 us, 32 of 25 tiles 52 and 40, 64 of
    // 8 tiles 33 and 36; 80 of 16 tiles 53 whole, 63 in two parts.
    if (2 * items > kSms || steps < 4) return 1;
    return (int)std::min<long long>(kSms / items, steps / 2);
}

int tc_dbias_splits(int B, int heads, int n, int m) {
    const long long items = (long long)heads * ((n + kRows - 1) / kRows) * ((m + kRows - 1) / kRows);
    // As above, over the batch, at least two entries to each part.  The backward from cold caches, whole and as here:
    // 4 items of 64 entries 102 and 53 us (46 in sixteen parts), 32 of 32 entries 92 and 70; 80 of 64 entries 237 whole,
    // 239 in two parts.
    if (2 * items > kSms || B < 4) return 1;
    return (int)std::min<long long>(kSms / items, B / 2);
}

cudaError_t launch_tc_backward(const Problem &p, int *err, cudaStream_t s) {
    Maps m;
    BwdParams x{};
    if (!fill_maps(m, x, p)) return cudaErrorInvalidValue;
    x.err = err;
    const int lut = offsets_smem(p.bias);
    const int keys = p.bias.mode == 2 ? round1k((p.m + 127) / 128 * 256) : 0;
    cudaError_t e;
    // ---- dQ and delta
    long long items = (long long)p.B * p.heads * x.qtiles;
    x.items = (int)items;
    x.first = 1;
    for (x.q_slots = 2;; --x.q_slots) {
        // with a bias the kernel holds 3728 bytes of its own
        const int left = kSmemBudget - (lut > 0 ? 1792 : 0) - 3 * x.q_slots * kTileBytes - lut - keys - 1024;
        x.stages = std::min(kMaxStages, left / (2 * kTileBytes));
        if (x.stages >= 2 || x.q_slots == 1) break;
    }
    if (x.stages < 2) return cudaErrorInvalidValue;   // a K tile is held until its dQ product, behind the next scores
    x.off_lut = (3 * x.q_slots + 2 * x.stages) * kTileBytes;
    x.off_aux = x.off_lut + lut;
    int bytes = x.off_aux + keys + 1024;
    e = p.bias.mode == 0   ? go_dq<tc_dq<0>>(m, x, bytes, s)
        : p.bias.mode == 1 ? go_dq<tc_dq<1>>(m, x, bytes, s)
                           : go_dq<tc_dq<2>>(m, x, bytes, s);
    if (e != cudaSuccess) return e;
    // ---- dK, dV
    items = (long long)p.B * p.kv_heads * x.ktiles * p.q_splits;
    x.items = (int)items;
    x.first = 0;
    x.splits = p.q_splits;
    x.div_splits = fast_div(x.splits);
    const int aux = (int)sizeof(QueryAux);
    for (x.q_slots = 2;; --x.q_slots) {
        const int left = kSmemBudget - 2 * x.q_slots * kTileBytes - kDkvOut - lut - 1024;
        x.stages = std::min(kMaxStages, left / (2 * kTileBytes + aux));
        if (x.stages >= 2 || x.q_slots == 1) break;
    }
    if (x.stages < 2) return cudaErrorInvalidValue;
    x.off_out = 2 * (x.q_slots + x.stages) * kTileBytes;
    x.off_lut = x.off_out + kDkvOut;
    x.off_aux = x.off_lut + lut;
    bytes = x.off_aux + x.stages * aux + 1024;
    e = p.bias.mode == 0   ? go<tc_dkdv<0>>(m, x, bytes, s)
        : p.bias.mode == 1 ? go<tc_dkdv<1>>(m, x, bytes, s)
                           : go<tc_dkdv<2>>(m, x, bytes, s);
    if (e != cudaSuccess) return e;
    if (p.q_splits > 1) {
        const size_t vecs = (size_t)p.B * p.kv_heads * p.m * (p.d / 4);
        e = launch_plain(join_dkdv, dim3((unsigned)((vecs + 255) / 256), 2), 256, 0, s, p);
        if (e != cudaSuccess) return e;
    }
    if (p.bias.mode == 0) return cudaSuccess;
    // ---- dS of the batch
    items = (long long)p.heads * x.qtiles * x.ktiles * p.b_splits;
    x.items = (int)items;
    x.splits = p.b_splits;
    x.div_splits = fast_div(x.splits);
    const int fold = kFoldTileBytes + (p.folded ? p.fold.units * 4 : 0);
    x.stages = std::min(kMaxStages, (kSmemBudget - fold - lut - 2048) / (4 * kTileBytes));
    if (x.stages < 1) return cudaErrorInvalidValue;
    x.off_out = 4 * x.stages * kTileBytes;
    x.off_lut = round1k(x.off_out + fold);
    x.off_aux = x.off_lut + lut;
    bytes = x.off_aux + 256 + 1024;
    return p.bias.mode == 1 ? go<tc_dbias<1>>(m, x, bytes, s) : go<tc_dbias<2>>(m, x, bytes, s);
}

}  // namespace attn
}  // namespace lisa
