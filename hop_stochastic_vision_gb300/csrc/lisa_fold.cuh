// lisa_fold.cuh -- sums of a 128 x 128 tile of pairs over the buckets of the
// relative position, for grids of the same spacing (key steps of 1).
//
// The tile is in shared memory.  All its pairs with one offset (dr, dc) lie on
// diagonals of the blocks that the grids' rows cut it into, so a thread owns an
// offset and walks them: neighbouring threads read neighbouring keys of one row
// (no bank conflict, no atomics, a fixed order).  The offsets' sums are then
// folded into the column buckets and left as one small block per tile,
// [offset rows][columns]; a second kernel adds the tiles up.  The matrix itself
// never goes to memory.
#pragma once

#include <cuda_runtime.h>

#include "lisa_attn.h"
#include "lisa_bias_dev.cuh"

namespace lisa {
namespace attn {
namespace {

constexpr int kFoldTile = 128;
constexpr int kFoldPitch = 133;       // floats: neighbouring rows 5 banks apart, diagonals 6, so a warp meets no
                                      // bank twice whether its lanes stand in one row or in one column
constexpr int kFoldTileBytes = kFoldTile * kFoldPitch * 4;

struct TileGeom {
    int q0, j0, nq, nk;
    int rq0, rq1, rk0, rk1;
    int dr_lo, dr_n;       // row differences rk - rq
    int dc_lo, dc_n;       // column differences ck - cq
    int cb_lo, cb_n;       // column buckets
};

__device__ __forceinline__ TileGeom fold_geom(const FoldDev &f, int it, int jt) {
    TileGeom g;
    g.q0 = it * kFoldTile;
    g.j0 = jt * kFoldTile;
    g.nq = min(kFoldTile, f.n - g.q0);
    g.nk = min(kFoldTile, f.m - g.j0);
    int c0 = g.q0, c1 = g.q0 + g.nq - 1, e0 = g.j0, e1 = g.j0 + g.nk - 1;
    g.rq0 = split(c0, f.div_q);
    g.rq1 = split(c1, f.div_q);
    g.rk0 = split(e0, f.div_k);
    g.rk1 = split(e1, f.div_k);
    if (g.rq0 != g.rq1) { c0 = 0; c1 = (int)f.div_q.d - 1; }
    if (g.rk0 != g.rk1) { e0 = 0; e1 = (int)f.div_k.d - 1; }
    g.dr_lo = g.rk0 - g.rq1;
    g.dr_n = g.rk1 - g.rq0 - g.dr_lo + 1;
    g.dc_lo = e0 - c1;
    g.dc_n = e1 - c0 - g.dc_lo + 1;
    if (f.cols.log_rule) {
        g.cb_lo = 0;
        g.cb_n = f.col_buckets;
    } else {
        const int D = f.cols.D, lo = g.dc_lo - f.start_c, hi = lo + g.dc_n - 1;
        g.cb_lo = min(max(lo, -D), D) + D;
        g.cb_n = min(max(hi, -D), D) + D - g.cb_lo + 1;
    }
    return g;
}

// u / d for 0 <= u < 2^15, d < 2^12: (u + 1/2) / d is at least 1 / (2 d) > 2^-13 from a whole number, far more than
// the product's rounding.
__device__ __forceinline__ int small_div(int u, float inv) { return (int)(((float)u + 0.5f) * inv); }

// Whether every offset of the tile is a column bucket of its own.
__device__ __forceinline__ bool fold_direct(const FoldDev &f, const TileGeom &g) {
    return !f.cols.log_rule && g.cb_n == g.dc_n;
}

// Sums of the tile's offsets, dr_n rows of dc_n, `pitch` apart; `threads` threads.
__device__ __forceinline__ void fold_offsets(const FoldDev &f, const TileGeom &g, const float *tile, float *sums,
                                             int pitch, int tid, int threads) {
    const int wq = (int)f.div_q.d, wk = (int)f.div_k.d;
    const float inv = 1.f / (float)g.dc_n;
    for (int u = tid; u < g.dr_n * g.dc_n; u += threads) {
        const int dri = small_div(u, inv), dr = g.dr_lo + dri, dc = g.dc_lo + (u - dri * g.dc_n);
        float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int rq = max(g.rq0, g.rk0 - dr); rq <= min(g.rq1, g.rk1 - dr); ++rq) {
            const int qb = rq * wq - g.q0, kb = (rq + dr) * wk - g.j0;   // tile row of cq = 0, column of ck = 0
            const int lo = max(max(0, -qb), max(0, -kb) - dc);
            const int hi = min(min(wq - 1, g.nq - 1 - qb), min(wk - 1, g.nk - 1 - kb) - dc);
            const float *p = tile + (qb + lo) * kFoldPitch + kb + lo + dc;
            int c = lo;
            for (; c + 7 <= hi; c += 8, p += 8 * (kFoldPitch + 1)) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = p[e * (kFoldPitch + 1)];
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] += v[e];
            }
            if (c <= hi) {   // the rest side by side too (64 x 64 grid step 376 us, 380 one by one)
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = c + e <= hi ? p[e * (kFoldPitch + 1)] : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] += v[e];
            }
        }
        sums[dri * pitch + (u - dri * g.dc_n)] = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
    }
}

// The offsets' sums into the tile's block of column buckets, [dr_n][f.K]; a warp
// per bucket (far buckets hold up to 255 offsets).
__device__ __forceinline__ void fold_buckets(const FoldDev &f, const TileGeom &g, const float *sums, float *out, int tid,
                                             int threads) {
    const int lane = tid & 31, total = g.dr_n * g.cb_n;
    const float inv = 1.f / (float)g.cb_n;
    for (int u = tid >> 5; u < total; u += threads >> 5) {
        const int dri = small_div(u, inv), c = u - dri * g.cb_n;
        int lo, hi;
        bucket_range(f.cols, g.cb_lo + c, lo, hi);
        lo = max(lo + f.start_c - g.dc_lo, 0);
        hi = min(hi + f.start_c - g.dc_lo, g.dc_n - 1);
        float s = 0.f;
        for (int x = lo + lane; x <= hi; x += 32) s += sums[dri * g.dc_n + x];
        if (hi - lo >= 1) {   // the same for the whole warp
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
        }
        if (lane == 0) out[dri * f.K + c] = s;
    }
}

__device__ __forceinline__ float *fold_block(const FoldDev &f, int part, int h, int it, int jt) {
    return f.part + ((((size_t)part * f.heads + h) * f.qtiles + it) * f.ktiles + jt) * ((size_t)f.nR * f.K);
}

}  // namespace
}  // namespace attn
}  // namespace lisa
