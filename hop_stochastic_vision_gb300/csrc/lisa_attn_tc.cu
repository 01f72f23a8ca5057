// lisa_attn_tc.cu -- the forward cross attention on the tensor cores (bf16).
//
// A persistent CTA takes work items of 256 queries (two tiles of 128 rows) of
// one (batch, head) and walks the keys in tiles of 128:
//   warp 9        TMA: the queries, then a ring of K and V tiles
//   warps 8, 10   one thread each issues the products of tile 0, 1: S_t = Q_t K^T
//                 into tensor memory, then O_t += P_t V with P_t read from there
//                 (one warp for both tiles spent 2240 cycles on the waits and
//                 instructions of a pair of tiles whose products take 1024)
//   warps 0-3     softmax of tile 0, one thread per row: scores to registers,
//   warps 4-7     weights to tensor memory as bf16; the same for tile 1
// While one tile's scores are in the softmax the other's products run.
// S, P and O of both tiles fill the 512 columns of tensor memory, so S of the
// next keys can be issued as soon as the scores are in registers.
//
// The running maximum is kept only to within 2^8: O and the sum are rescaled
// when a tile's maximum passes the reference by more, which after the first
// tile is rare, so the accumulator stays in tensor memory.  exp is 2^x with
// log2(e) folded into the scale and into the bias table.
//
// 65536 queries on 1024 keys, 4 heads of 64: 77 us from cold caches, 890 TFLOP/s,
// 47% of the measured bf16 rate.  A 128 x 128 tile costs about 1300 cycles, 512 of
// products and 512 on the exponential unit; both are 42% busy.
#include <type_traits>

#include "lisa_attn_tc.cuh"

namespace lisa {
namespace attn {
namespace {

// 384 threads x 168 registers at launch = 2 x 128 x 208 + 128 x 88 after the split
constexpr int kFwdThreads = 384;
constexpr int kRegsSoftmax = 208, kRegsControl = 88;
constexpr int kMaxStages = 5;
constexpr float kSlack = 8.f;
constexpr float kFarRef = 0x1p24f;

struct FwdParams {
    Problem p;
    MapUse uq, uk, uv;
    int *err;
    int qtiles;      // pairs of 128 queries per (batch, head)
    int splits;
    int items;
    FastDiv div_splits, div_qtiles, div_B, div_group;
    int stages;
    int off_out, off_lut, off_keys;   // dynamic shared memory, behind Q and the ring
};

// Dynamic shared memory: the barriers and what else is static fit in 1 KB.  Behind the tiles come the softmax warps'
// staging blocks, the offsets (with the four zeros behind them) and the keys' offsets, packed: the largest grids' leave
// room for two stages with 992 bytes to spare.
constexpr int kFwdSmem = 226 * 1024;
constexpr int kStaging = 8 * 4096;
constexpr int offsets_bytes_smem(int entries) { return entries ? (entries * 4 + 32 + 15) / 16 * 16 : 0; }
constexpr int keys_bytes_smem(int m) { return (m + kRows - 1) / kRows * kRows * 2; }
static_assert((2 + 2 * 2) * kTileBytes + kStaging + offsets_bytes_smem(LISA_MAX_OFFSETS) +
                      keys_bytes_smem(LISA_MAX_OFFSETS) + 1024 <= kFwdSmem,
              "every bias that the argument checks accept has room for two stages");

struct FwdBars {
    uint64_t q_full[2], q_empty[2], k_full[kMaxStages], v_full[kMaxStages], k_empty[kMaxStages], v_empty[kMaxStages];
    uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], lut_full;
};

struct Item {
    int h, b, q0, split, len, t0, t1, nt;
};
__device__ __forceinline__ Item item_of(const FwdParams &x, int it) {
    Item w;
    int qt = split(it, x.div_splits);
    w.split = it;
    w.b = split(qt, x.div_qtiles);
    w.q0 = qt * 2 * kRows;
    w.h = split(w.b, x.div_B);
    w.len = keys_of(x.p, w.b);
    const int tiles = (w.len + kRows - 1) / kRows, per = quotient(tiles + x.splits - 1, x.div_splits);
    w.t0 = min(w.split * per, tiles);
    w.t1 = min(w.t0 + per, tiles);
    w.nt = x.p.n - w.q0 > kRows ? 2 : 1;
    return w;
}
// Valid keys of tile `t`, and the columns its products cover.
__device__ __forceinline__ int tile_keys(int len, int t) { return min(kRows, len - t * kRows); }
__device__ __forceinline__ int tile_cols(int keys) { return (keys + 15) & ~15; }

// A row's state over the tiles of an item, and what its bias needs.
struct RowState {
    float ref, sum;
    float limit;     // a maximum above it moves the reference: ref + kSlack, -inf where ref is far from 0
    int oq, oq_lo;
};

// Bias of N columns from key j0: s -> scale2 s + bias, or one value for all of
// them (2^(mul s + add) is what comes of it).
template <int kBias, int N>
__device__ __forceinline__ void add_bias(float (&s)[N], const BiasDev &b, const float *lut, const uint16_t *key_off,
                                         int j0, int keys, const RowState &r, float scale2, float &mul, float &add) {
    mul = scale2;
    add = 0.f;
    if (kBias == 1) {
        const int lo = b.step_c * j0 - r.oq_lo - 31, hi = b.step_c * (j0 + keys - 1) - r.oq_lo, last = b.entries - 1;
        if (hi <= 0 || lo >= last) {          // the whole tile in one outermost bucket
            add = lut[hi <= 0 ? 0 : last];
        } else {
            const int off = b.step_c * j0 - r.oq;
            mul = 1.f;
            if (b.step_c == 1) {   // inside the padded table
                const float *l = lut + off;
#pragma unroll
                for (int c = 0; c < N; ++c) s[c] = fmaf(s[c], scale2, l[c]);
            } else {
#pragma unroll
                for (int c = 0; c < N; ++c) s[c] = fmaf(s[c], scale2, lut[min(max(off + b.step_c * c, 0), last)]);
            }
        }
    } else if (kBias == 2) {
        // inside the table by construction (key_off repeats the last key behind the end)
        mul = 1.f;
        grid_bias(s, b, lut - r.oq, key_off, j0, scale2);
    }
}

template <int kBias>
__global__ void __launch_bounds__(kFwdThreads, 1)
    tc_forward(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ FwdParams x) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);   // stays a shared-memory pointer
    __shared__ __align__(8) FwdBars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    const Problem &p = x.p;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = smem_u32(sm);
    const uint32_t q_smem = base, ring = base + 2 * kTileBytes;
    float *lut = reinterpret_cast<float *>(sm + x.off_lut) + p.bias.pad;
    uint16_t *key_off = reinterpret_cast<uint16_t *>(sm + x.off_keys);
    const Guard guard{x.err, &dead};

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bar.q_full[t]), 1);
            mbar_init(smem_u32(&bar.q_empty[t]), 1);
            mbar_init(smem_u32(&bar.s_full[t]), 1);
            mbar_init(smem_u32(&bar.s_free[t]), 4);
            mbar_init(smem_u32(&bar.p_full[t]), 4);
            mbar_init(smem_u32(&bar.pv_done[t]), 1);
        }
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(smem_u32(&bar.k_full[s]), 1);
            mbar_init(smem_u32(&bar.v_full[s]), 1);
            mbar_init(smem_u32(&bar.k_empty[s]), 2);   // one for each tile
            mbar_init(smem_u32(&bar.v_empty[s]), 2);
        }
        mbar_init(smem_u32(&bar.lut_full), 1);
        dead = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(smem_u32(&tmem_slot), 512);
    if (kBias == 2)
        for (int j = tid; j < (p.m + 127) / 128 * 128; j += kFwdThreads) key_off[j] = (uint16_t)off_key(p.bias, min(j, p.m - 1));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    chain_begin();
    if (blockIdx.x == 0 && tid == 0) *x.err = 0;

    if (warp >= 8) set_regs_down<kRegsControl>();
    if (warp == 11) {
        // idle: completes the control warps' group of four
    } else if (warp == 9) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int kt = 0, nq[2] = {0, 0};
            Cursor c;
            for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
                const Item w = item_of(x, it);
                if (w.t0 >= w.t1) continue;
                auto load_q = [&](int t) {
                    const uint32_t f = smem_u32(&bar.q_full[t]);
                    if (nq[t] > 0) wait_on(smem_u32(&bar.q_empty[t]), (nq[t] - 1) & 1, guard, kErrTimeoutMma);
                    mbar_arrive_expect_tx(f, kTileBytes);
                    load_rows(q_smem + t * kTileBytes, &mq, x.uq, w.q0 + t * kRows, w.h, w.b, f);
                    ++nq[t];
                };
                load_q(0);
                const int g = quotient(w.h, x.div_group);
                for (int j = w.t0; j < w.t1; ++j, ++kt, c.next(x.stages)) {
                    const int s = c.slot;
                    const uint32_t kf = smem_u32(&bar.k_full[s]), vf = smem_u32(&bar.v_full[s]);
                    if (kt >= x.stages) wait_on(smem_u32(&bar.k_empty[s]), c.phase ^ 1u, guard, kErrTimeoutMma);
                    mbar_arrive_expect_tx(kf, kTileBytes);
                    load_rows(ring + 2 * s * kTileBytes, &mk, x.uk, j * kRows, g, w.b, kf);
                    if (j == w.t0 && w.nt == 2) load_q(1);
                    if (kt >= x.stages) wait_on(smem_u32(&bar.v_empty[s]), c.phase ^ 1u, guard, kErrTimeoutMma);
                    mbar_arrive_expect_tx(vf, kTileBytes);
                    load_rows(ring + (2 * s + 1) * kTileBytes, &mv, x.uv, j * kRows, g, w.b, vf);
                }
            }
            // nothing may still arrive on this CTA's barriers once it has gone
            for (int s = 0; s < x.stages; ++s) {
                const int uses = kt > s ? (kt - 1 - s) / x.stages + 1 : 0;
                if (uses == 0) continue;
                if (!mbar_wait(smem_u32(&bar.k_empty[s]), (uses - 1) & 1) ||
                    !mbar_wait(smem_u32(&bar.v_empty[s]), (uses - 1) & 1))
                    atomicOr(x.err, kErrTimeoutMma);
            }
            for (int t = 0; t < 2; ++t)
                if (nq[t] > 0 && !mbar_wait(smem_u32(&bar.q_empty[t]), (nq[t] - 1) & 1))
                    atomicOr(x.err, kErrTimeoutMma);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // --------------------------------------------------------- products
        const int t = warp == 8 ? 0 : 1;
        const uint32_t tS = tmem + t * 128, tP = tmem + 256 + t * 64, tO = tmem + 384 + t * 64;
        const uint64_t dq = desc_rows(q_smem + t * kTileBytes), dk = desc_rows(ring), dv = desc_tokens(ring + kTileBytes);
        constexpr uint32_t kPair = 2 * kTileBytes / 16;
        int nq = 0, ns = 0, np = 0;
        Cursor ck, cv;
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(x, it);
            if (w.t0 >= w.t1) continue;
            if (t >= w.nt) {   // no rows in this tile: pass its share of the ring on
                for (int j = w.t0; j < w.t1; ++j) {
                    wait_on(smem_u32(&bar.k_full[ck.slot]), ck.phase, guard, kErrTimeoutLoad);
                    wait_on(smem_u32(&bar.v_full[ck.slot]), ck.phase, guard, kErrTimeoutLoad);
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&bar.k_empty[ck.slot]));
                        mbar_arrive(smem_u32(&bar.v_empty[ck.slot]));
                    }
                    ck.next(x.stages);
                }
                cv = ck;
                continue;
            }
            wait_on(smem_u32(&bar.q_full[t]), nq++ & 1, guard, kErrTimeoutLoad);
            auto scores = [&](int j) __attribute__((always_inline)) {
                wait_on(smem_u32(&bar.k_full[ck.slot]), ck.phase, guard, kErrTimeoutLoad);
                if (ns > 0) wait_on(smem_u32(&bar.s_free[t]), (ns - 1) & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                if (elect_one()) {
                    mma_rows_rows(tS, dq, dk + (uint32_t)ck.slot * kPair, tile_cols(tile_keys(w.len, j)));
                    tc_commit(smem_u32(&bar.s_full[t]));
                    tc_commit(smem_u32(&bar.k_empty[ck.slot]));
                    if (j == w.t1 - 1) tc_commit(smem_u32(&bar.q_empty[t]));
                }
                __syncwarp();
                ++ns;
                ck.next(x.stages);
            };
            scores(w.t0);
            for (int j = w.t0; j < w.t1; ++j) {
                if (j + 1 < w.t1) scores(j + 1);
                wait_on(smem_u32(&bar.v_full[cv.slot]), cv.phase, guard, kErrTimeoutLoad);
                wait_on(smem_u32(&bar.p_full[t]), np & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                if (elect_one()) {
                    mma_weights_rows(tO, tP, dv + (uint32_t)cv.slot * kPair, tile_cols(tile_keys(w.len, j)), j > w.t0);
                    tc_commit(smem_u32(&bar.pv_done[t]));
                    tc_commit(smem_u32(&bar.v_empty[cv.slot]));
                }
                __syncwarp();
                ++np;
                cv.next(x.stages);
            }
        }
    } else {
        // ---------------------------------------------------------- softmax
        set_regs_up<kRegsSoftmax>();
        const int t = warp >> 2, wt = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // 32 lanes per warp
        const uint32_t s_tm = tmem + t * 128 + lanes, p_tm = tmem + 256 + t * 64 + lanes, o_tm = tmem + 384 + t * 64 + lanes;
        const float scale2 = p.scale * kLog2e;
        int kt = 0, ns = 0, np = 0, lut_head = -1, luts = 0;
        for (int it = blockIdx.x; it < x.items; it += gridDim.x) {
            const Item w = item_of(x, it);
            if (kBias && w.h != lut_head) {
                load_offsets<256>(p.bias, w.h, lut, &bar.lut_full, luts, tid, guard);
                lut_head = w.h;
            }
            if (t >= w.nt) {   // this tile has no rows
                kt += w.t1 - w.t0;
                continue;
            }
            const int i = w.q0 + t * kRows + wt;
            RowState r{-INFINITY, 0.f, -INFINITY, 0, 0};
            if (kBias) {
                const int start = bias_start(p.bias, w.b);
                r.oq = off_query(p.bias, kBias == 2 ? min(i, p.n - 1) : i, start);
                r.oq_lo = off_query(p.bias, i - lane, start);   // sequence: the warp's first row
            }
            // a whole tile (N = 0), a part of one, a part of at most 64 keys
            auto tile = [&](int j, auto variant) __attribute__((always_inline)) {
                constexpr bool kFull = decltype(variant)::value == 0;
                constexpr int N = kFull ? kRows : decltype(variant)::value;
                const int keys = kFull ? kRows : tile_keys(w.len, j), cols = kFull ? kRows : tile_cols(keys), j0 = j * kRows;
                float s[N];
                wait_on(smem_u32(&bar.s_full[t]), ns & 1, guard, kErrTimeoutMma);
                ++ns;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < N; c += 32) tmem_ld32_nowait(s_tm + c, s + c);
                tc_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar.s_free[t]));

                float mul, add;   // 2^(mul s + add - ref) is the weight
                add_bias<kBias, N>(s, p.bias, lut, key_off, j0, keys, r, scale2, mul, add);
                if (!kFull) {
#pragma unroll
                    for (int c = 0; c < N; ++c)
                        if (c >= keys) s[c] = -INFINITY;
                }
                float top;
                {
                    float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int c = 4; c < N; c += 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            m4[e] = c + e + 4 < N ? fmaxf(fmaxf(m4[e], s[c + e]), s[c + e + 4]) : fmaxf(m4[e], s[c + e]);
                    }
                    top = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), mul, add);
                }
                const bool first = j == w.t0;
                // The maximum's rounding in `ref` is a power of two common to the row's weights and goes out with the sum
                // while it is small.  Further out (half a unit in the last place of 2^24 is 1, of 2^33 is 512) the scores
                // are rounded as the maximum was, in every tile, so that the largest weight is 2^0 whatever their size.
                auto refer = [&](float now) __attribute__((always_inline)) {
                    r.ref = now;
                    const bool far = fabsf(now) > kFarRef;
                    r.limit = far ? -INFINITY : now + kSlack;
                    if (kBias != 2 && __any_sync(0xFFFFFFFFu, far)) {
#pragma unroll
                        for (int c = 0; c < N; ++c) s[c] = fmaf(s[c], mul, add);
                        mul = 1.f;
                        add = 0.f;
                    }
                };
                if (first) {
                    refer(top);
                } else if (__any_sync(0xFFFFFFFFu, top > r.limit)) {
                    const float now = fmaxf(r.ref, top);
                    const float f = r.ref == -INFINITY ? 0.f : ex2_approx(r.ref - now);
                    refer(now);
                    r.sum *= f;
                    wait_on(smem_u32(&bar.pv_done[t]), (np - 1) & 1, guard, kErrTimeoutMma);
                    tc_fence_after();
                    float o[32];
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        tmem_ld32_nowait(o_tm + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tmem_st32(o_tm + c, o);
                    }
                    tc_wait_st();
                }
                const float shift = add - (r.ref == -INFINITY ? 0.f : r.ref);   // a row of -inf so far: weights 0, not NaN
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                // the previous weights have been read (and their products are in O)
                if (!first) wait_on(smem_u32(&bar.pv_done[t]), (np - 1) & 1, guard, kErrTimeoutMma);
#pragma unroll
                for (int c = 0; c < N; c += 32)
                    if (kFull || c < cols) {
                        uint32_t w16[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a, b;
                            fma2(a, b, s[c + e], s[c + e + 1], mul, mul, shift, shift);
                            a = ex2_approx(a);
                            b = ex2_approx(b);
                            add2(part[e & 2], part[(e & 2) + 1], part[e & 2], part[(e & 2) + 1], a, b);
                            w16[e >> 1] = pack_bf16(a, b);
                        }
                        tmem_st16(p_tm + c / 2, w16);
                    }
                r.sum += (part[0] + part[1]) + (part[2] + part[3]);
                if (!kFull && keys < cols && w.len < p.m) {
                    // values behind the last key: whatever stands there times a weight of 0 has to be 0
                    // (for each tile's own product; the second time zeros meet zeros)
                    const int st = kt % x.stages;
                    wait_on(smem_u32(&bar.v_full[st]), (kt / x.stages) & 1, guard, kErrTimeoutLoad);
                    zero_rows(ring + (2 * st + 1) * kTileBytes, keys, cols, wt);
                    fence_proxy_async();
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar.p_full[t]));
                ++np;
                ++kt;
            };
            for (int j = w.t0; j < w.t1; ++j) {
                const int keys = tile_keys(w.len, j);
                if (keys == kRows)
                    tile(j, std::integral_constant<int, 0>{});
                else if (keys > 64)
                    tile(j, std::integral_constant<int, 128>{});
                else
                    tile(j, std::integral_constant<int, 64>{});
            }
            const float ref = r.ref, sum = r.sum;
            // ------------------------------------------------------ output
            float o[64];
            if (w.t0 < w.t1) {
                wait_on(smem_u32(&bar.pv_done[t]), (np - 1) & 1, guard, kErrTimeoutMma);
                tc_fence_after();
                tmem_ld32_nowait(o_tm, o);
                tmem_ld32_nowait(o_tm + 32, o + 32);
                tc_wait_ld();
                tc_fence_before();
            } else {
#pragma unroll
                for (int c = 0; c < 64; ++c) o[c] = 0.f;
            }
            const float inv = sum != 0.f ? 1.f / sum : 0.f;
            const float lse = ref == -INFINITY ? -INFINITY : kLn2 * (ref + log2f(sum));
            const size_t row = ((size_t)w.b * p.heads + w.h) * p.n + i;
            if (x.splits == 1) {
                const int i0 = i - lane;
                store_rows_bf16<64>(base + x.off_out + (uint32_t)warp * 4096u, o, inv,
                                    static_cast<__nv_bfloat16 *>(const_cast<void *>(p.O.p)) + (long long)w.b * p.O.sb +
                                        (long long)w.h * p.O.sh + (long long)i0 * p.O.st,
                                    p.O.st, p.n - i0, p.d, lane);
                if (p.lse && i < p.n) p.lse[row] = lse;
            } else if (i < p.n) {
                const size_t at = (size_t)w.split * ((size_t)p.B * p.heads * p.n) + row;
                p.stat_part[at] = make_float2(ref, sum);
                float4 *op = reinterpret_cast<float4 *>(p.o_part + at * p.d);
#pragma unroll
                for (int c = 0; c < 64; c += 4)
                    if (c < p.d) op[c / 4] = make_float4(o[c] * inv, o[c + 1] * inv, o[c + 2] * inv, o[c + 3] * inv);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// o = sum_s w_s o_s / sum_s w_s with w_s = 2^(ref_s - ref) sum_s: the parts of a row, in order.  Reference and sum come
// apart: far from 0 their lse would have lost the sum (at 2^24 the last place is 2), and parts of unequal lengths would
// weigh the same.
__global__ void __launch_bounds__(256) join_splits(const __grid_constant__ Problem p) {
    chain_begin();
    const int vec = p.d / 4;
    const size_t rows = (size_t)p.B * p.heads * p.n;
    const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
    const size_t row = at / vec;
    const int c = (int)(at % vec) * 4;
    if (row >= rows) return;
    float top = -INFINITY;
    for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.stat_part[s * rows + row].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.splits; ++s) {
        const float2 st = p.stat_part[s * rows + row];
        const float w = ex2_approx(st.x - ref) * st.y;
        const float4 v = *reinterpret_cast<const float4 *>(p.o_part + (s * rows + row) * p.d + c);
        sum += w;
        o[0] = fmaf(w, v.x, o[0]);
        o[1] = fmaf(w, v.y, o[1]);
        o[2] = fmaf(w, v.z, o[2]);
        o[3] = fmaf(w, v.w, o[3]);
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const int i = (int)(row % p.n), h = (int)(row / p.n % p.heads);
    const long long b = (long long)(row / p.n / p.heads);
    const long long out = b * p.O.sb + (long long)h * p.O.sh + (long long)i * p.O.st + c;
    uint2 r;
    r.x = pack_bf16(o[0] * inv, o[1] * inv);
    r.y = pack_bf16(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(const_cast<void *>(p.O.p)) + out) = r;
    if (c == 0 && p.lse) p.lse[row] = top == -INFINITY ? -INFINITY : kLn2 * (top + log2f(sum));
}

// Joins p.splits partial outputs (o_part, stat_part) into O and lse.
cudaError_t launch_join(const Problem &p, cudaStream_t s) {
    const size_t vecs = (size_t)p.B * p.heads * p.n * (p.d / 4);
    return launch_chained(join_splits, dim3((unsigned)((vecs + 255) / 256)), 256, 0, s, p);
}

}  // namespace

int tc_forward_splits(int B, int heads, int n, int m) {
    const long long items = (long long)B * heads * ((n + 2 * kRows - 1) / (2 * kRows));
    const int tiles = (m + kRows - 1) / kRows;
    // Fewer items than half the SMs: share the keys out in one round, at least two tiles to each part (the parts' outputs
    // go through memory).  From cold caches, whole and as here: one item of 32 tiles 42 and 22 us, 16 items of 32 tiles 42
    // and 26, 48 of 16 tiles 28 and 26, 72 of 16 tiles 28 and 30.  Fewer parts would do better where one
    // item has 256 tiles: whole 256 us, 128 parts as here 61, 32 parts 34.
    if (items * 2 > kSms || tiles < 4) return 1;
    return (int)std::min<long long>(kSms / items, tiles / 2);
}

cudaError_t launch_tc_forward(const Problem &p, int *err, cudaStream_t s) {
    FwdParams x{};
    x.p = p;
    x.err = err;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, &x.uq, p.Q, p.B, p.heads, p.n, p.d) || !make_map(&mk, &x.uk, p.K, p.B, p.kv_heads, p.m, p.d) ||
        !make_map(&mv, &x.uv, p.V, p.B, p.kv_heads, p.m, p.d))
        return cudaErrorInvalidValue;
    x.qtiles = (p.n + 2 * kRows - 1) / (2 * kRows);
    x.splits = p.splits;
    const long long items = (long long)p.B * p.heads * x.qtiles * x.splits;
    x.items = (int)items;
    x.div_splits = fast_div(x.splits);
    x.div_qtiles = fast_div(x.qtiles);
    x.div_B = fast_div(p.B);
    x.div_group = fast_div(p.group);
    const int lut = offsets_bytes_smem(p.bias.mode ? p.bias.entries + 2 * p.bias.pad : 0);
    const int keys = p.bias.mode == 2 ? keys_bytes_smem(p.m) : 0;
    const int fixed = 2 * kTileBytes + kStaging + lut + keys + 1024;
    const int tiles = (p.m + kRows - 1) / kRows;
    x.stages = std::min(std::min(kMaxStages, (kFwdSmem - fixed) / (2 * kTileBytes)), std::max(2, tiles + 1));
    x.off_out = (2 + 2 * x.stages) * kTileBytes;
    x.off_lut = x.off_out + kStaging;
    x.off_keys = x.off_lut + lut;
    const int bytes = x.off_keys + keys + 1024;
    const unsigned grid = (unsigned)std::min(x.items, sms());
    cudaError_t e;
    switch (p.bias.mode) {
        case 0:
            if ((e = allow_smem<tc_forward<0>>()) == cudaSuccess)
                e = launch_chained(tc_forward<0>, grid, kFwdThreads, bytes, s, mq, mk, mv, x);
            break;
        case 1:
            if ((e = allow_smem<tc_forward<1>>()) == cudaSuccess)
                e = launch_chained(tc_forward<1>, grid, kFwdThreads, bytes, s, mq, mk, mv, x);
            break;
        default:
            if ((e = allow_smem<tc_forward<2>>()) == cudaSuccess)
                e = launch_chained(tc_forward<2>, grid, kFwdThreads, bytes, s, mq, mk, mv, x);
    }
    if (e == cudaSuccess && p.splits > 1) e = launch_join(p, s);
    return e;
}

}  // namespace attn
}  // namespace lisa
