// lisa_attn_tc.cuh -- pieces shared by the tensor-core kernels of the cross
// attention (bf16): bounded waits that give up once per CTA, tensor-memory
// transfers of whole rows, packed fp32 arithmetic, tensor maps of strided
// [B][heads][tokens][d] tensors.
//
// Head widths 16 and 32 use the kernels of 64: their tiles are loaded with a
// 64-wide box over a narrower tensor, so TMA fills columns d .. 63 with zeros,
// which add nothing to any product; only d columns are stored.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lisa_attn.h"
#include "lisa_bias_dev.cuh"
#include "lisa_internal.h"
#include "lisa_launch.cuh"
#include "lisa_tc_common.cuh"

namespace lisa {
namespace attn {
namespace {

using namespace lisa::sm100;

constexpr int kRows = 128;                    // rows of a tile: queries or keys
constexpr int kTileBytes = kRows * 128;       // 128 tokens x 64 bf16
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A CTA whose wait gave up stops waiting altogether (its results are undefined
// and the error word says so), so a failure costs one limit, not one per wait.
struct Guard {
    int *err;
    volatile int *dead;
};
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void wait_on(uint32_t bar, uint32_t parity, const Guard &g, int bit) {
    if (phase_done(bar, parity)) return;
    const long long t0 = clock64();
    while (!mbar_test_parity_suspend(bar, parity)) {
        if (*g.dead) return;
        if (clock64() - t0 > kWaitCycles) {
            atomicOr(g.err, bit);
            *g.dead = 1;
            return;
        }
    }
}

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, float *r) {
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
          "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, float *r) {
    tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(r));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float *r) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(r);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
        "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
        "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}
// Registers of this warpgroup's threads, out of what the block was launched with.
template <int N>
__device__ __forceinline__ void set_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations in one instruction, on neighbouring registers.
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b, float c, float d, float e, float f) {
    // (x, y) = (a, b) * (c, d) + (e, f)
    asm("{\n.reg .b64 p, q, r;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\nmov.b64 r, {%6, %7};\n"
        "fma.rn.f32x2 p, p, q, r;\nmov.b64 {%0, %1}, p;\n}"
        : "=f"(x), "=f"(y)
        : "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f));
}
__device__ __forceinline__ void add2(float &x, float &y, float a, float b, float c, float d) {
    asm("{\n.reg .b64 p, q;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\n"
        "add.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}"
        : "=f"(x), "=f"(y)
        : "f"(a), "f"(b), "f"(c), "f"(d));
}
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b, float c, float d) {
    asm("{\n.reg .b64 p, q;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\n"
        "mul.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}"
        : "=f"(x), "=f"(y)
        : "f"(a), "f"(b), "f"(c), "f"(d));
}

// D[tmem] (+)= A[tmem] * B[smem]: A's rows are the 128 lanes, two bf16 of a row per 32-bit column.
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptors of a token tile (128-byte rows, 128-byte swizzle): its rows as the
// M or N side of a product over d (K-major), or as the K side of a product over
// tokens (MN-major).  One thread issues every product, so the steps along K are
// additions to a descriptor and the loops are unrolled: building a descriptor
// for each instruction took 80 cycles of that thread per instruction, three
// times what the instruction itself takes.
__device__ __forceinline__ uint64_t desc_rows(uint32_t tile) { return make_desc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t desc_tokens(uint32_t tile) { return make_desc_sw128(tile, 1024, 1024); }

// One thread of a converged warp, the same one every time.  The warp runs the
// loops and waits as a whole and only the products and commits are under this:
// addresses and descriptors then stay in uniform registers, where the
// instructions want them.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred e;\nelect.sync _|e, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, e;\n}" : "=r"(p));
    return p != 0;
}

// [128 x cols] = A (tile of 128 rows) * B^T (tile of >= cols rows); K = 64.
__device__ __forceinline__ void mma_rows_rows(uint32_t d_tmem, uint64_t a, uint64_t b, int cols) {
    const uint32_t idesc = make_idesc_bf16(128, 0, false, false) | ((uint32_t)(cols >> 3) << 17);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) tc_mma(d_tmem, a + 2 * ks, b + 2 * ks, idesc, ks > 0);
}
// [128 x 64] (+)= A (tensor memory, 128 x k) * B (tile of k token rows); k a multiple of 16.
__device__ __forceinline__ void mma_weights_rows(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, int k,
                                                 bool accumulate) {
    constexpr uint32_t idesc = make_idesc_bf16(128, 64, false, true);
    if (k == 128) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) tc_mma_ta(d_tmem, a_tmem + ks * 8, b + 128 * ks, idesc, ks > 0 || accumulate);
    } else {
        for (int ks = 0; ks < k / 16; ++ks)
            tc_mma_ta(d_tmem, a_tmem + ks * 8, b + 128 * ks, idesc, ks > 0 || accumulate);
    }
}

// A position in a ring of `stages` slots.
struct Cursor {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// The head's offset table (bias_offsets: fp32, log2(e) folded in) by one bulk
// copy.  Called by the kThreads arithmetic threads together; `count` copies so far.
template <int kThreads>
__device__ __forceinline__ void load_offsets(const BiasDev &b, int head, float *lut, uint64_t *bar, int &count, int tid,
                                             const Guard &g) {
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");   // every warp is past its reads of the old table
    if (tid == 0) {
        fence_proxy_async();
        const uint32_t bytes = (uint32_t)(b.entries + 2 * b.pad + 4 + 3) / 4 * 16;
        mbar_arrive_expect_tx(smem_u32(bar), bytes);
        bulk_load(smem_u32(lut - b.pad), b.offsets + (size_t)head * b.offsets_pitch, bytes, smem_u32(bar));
    }
    wait_on(smem_u32(bar), count & 1, g, kErrTimeoutLoad);
    ++count;
}

// s[c] = scale2 s[c] + bias of N keys from `j0` (grids): key_off holds each key's
// offset, `l` points at the row's own.  Where a grid's rows are multiples of four
// keys wide, one offset serves four neighbouring values.
template <int N>
__device__ __forceinline__ void grid_bias(float (&s)[N], const BiasDev &b, const float *l, const uint16_t *key_off, int j0,
                                          float scale2) {
    if (b.run_k) {
#pragma unroll
        for (int c = 0; c < N; c += 4) {
            const float *v = l + key_off[j0 + c];
            s[c] = fmaf(s[c], scale2, v[0]);
            s[c + 1] = fmaf(s[c + 1], scale2, v[1]);
            s[c + 2] = fmaf(s[c + 2], scale2, v[2]);
            s[c + 3] = fmaf(s[c + 3], scale2, v[3]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 4) {
            const uint2 a = *reinterpret_cast<const uint2 *>(key_off + j0 + c);
            s[c] = fmaf(s[c], scale2, l[a.x & 0xFFFFu]);
            s[c + 1] = fmaf(s[c + 1], scale2, l[a.x >> 16]);
            s[c + 2] = fmaf(s[c + 2], scale2, l[a.y & 0xFFFFu]);
            s[c + 3] = fmaf(s[c + 3], scale2, l[a.y >> 16]);
        }
    }
}

// One token box {64, 128} of a head's slice; coordinates of repeated dimensions stay 0.
struct MapUse {
    int hmul, bmul;
};
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *m, const MapUse &u, int token, int head,
                                          int batch, uint32_t bar) {
    tma_load_4d(dst, m, 0, token, head * u.hmul, batch * u.bmul, bar);
}

// Zeroes rows r0 .. r1 - 1 (at most 15) of a token tile; all 128 threads of a warpgroup.
__device__ __forceinline__ void zero_rows(uint32_t tile, int r0, int r1, int t) {
    const int row = r0 + (t >> 3);
    if (row < r1) st_shared_v4(tile + (uint32_t)row * 128u + (uint32_t)(t & 7) * 16u, 0, 0, 0, 0);
}

__device__ __forceinline__ int keys_of(const Problem &p, int b) {
    return p.kv_lens ? min(max(p.kv_lens[b], 0), p.m) : p.m;
}

// 32 rows of a warp, one per lane, to bf16 in memory: through 4 KB of the warp's
// own shared memory, so that a store instruction writes whole rows (a store per
// lane and row touches 32 lines each time: 2000 cycles for a tile).
//   COLS  columns of a lane's row (64 or 32), of which columns < d exist
//   row0  address of lane 0's row; rows `stride` elements apart, `rows` of them exist
template <int COLS>
__device__ __forceinline__ void store_rows_bf16(uint32_t stage, const float *v, float mul, __nv_bfloat16 *row0,
                                                long long stride, int rows, int d, int lane) {
    constexpr int kChunks = COLS / 8;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
        st_shared_v4(stage + (uint32_t)lane * (COLS * 2) + (uint32_t)((c ^ (lane & (kChunks - 1))) << 4),
                     pack_bf16(v[8 * c] * mul, v[8 * c + 1] * mul), pack_bf16(v[8 * c + 2] * mul, v[8 * c + 3] * mul),
                     pack_bf16(v[8 * c + 4] * mul, v[8 * c + 5] * mul), pack_bf16(v[8 * c + 6] * mul, v[8 * c + 7] * mul));
    __syncwarp();
    const int c = lane % kChunks, r0 = lane / kChunks;
    row0 += r0 * stride + 8 * c;
    const long long step = (32 / kChunks) * stride;
    const int last = 8 * c < d ? rows : 0;
#pragma unroll
    for (int e = 0; e < kChunks; ++e, row0 += step) {
        const int r = e * (32 / kChunks) + r0;
        if (r < last) {
            uint4 o;
            ld_shared_v4(stage + (uint32_t)r * (COLS * 2) + (uint32_t)((c ^ (r & (kChunks - 1))) << 4), o.x, o.y, o.z, o.w);
            *reinterpret_cast<uint4 *>(row0) = o;
        }
    }
    __syncwarp();
}

// ---------------------------------------------------------------- host side
// 4-D map {d, tokens, heads, B} of a strided bf16 tensor, box {64, 128, 1, 1}.
inline bool make_map(CUtensorMap *m, MapUse *u, const Tensor &t, int B, int heads, int tokens, int d) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    u->hmul = heads > 1 && t.sh > 0 ? 1 : 0;
    u->bmul = B > 1 && t.sb > 0 ? 1 : 0;
    const cuuint64_t row = (cuuint64_t)(tokens > 1 ? t.st : d) * 2;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)tokens, (cuuint64_t)(u->hmul ? heads : 1),
                          (cuuint64_t)(u->bmul ? B : 1)};
    cuuint64_t strides[3] = {row, u->hmul ? (cuuint64_t)t.sh * 2 : row, u->bmul ? (cuuint64_t)t.sb * 2 : row};
    cuuint32_t box[4] = {64, kRows, 1, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(t.p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int sms() {
    static std::atomic<int> n[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    int v = n[dev].load(std::memory_order_relaxed);
    if (v == 0) n[dev].store(v = sm_count(), std::memory_order_relaxed);
    return v;
}

constexpr int kSmemBudget = 227 * 1024 - 2048;   // dynamic: behind the barriers

// Shared memory of a head's offsets.
inline int offsets_smem(const BiasDev &b) { return b.mode ? ((b.entries + 2 * b.pad) * 4 + 32 + 1023) / 1024 * 1024 : 0; }

inline int round1k(int x) { return (x + 1023) / 1024 * 1024; }

}  // namespace
}  // namespace attn
}  // namespace lisa
