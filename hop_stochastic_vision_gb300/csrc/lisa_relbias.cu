// lisa_relbias.cu -- the relative position bias as a matrix, and its gradient.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lisa_attn.h"
#include "lisa_bias_dev.cuh"
#include "lisa_fold.cuh"
#include "lisa_launch.cuh"

namespace lisa {
namespace attn {
namespace {

constexpr int kDenseThreads = 256;
// Offsets of a tile that are folded in shared memory: three CTAs of fold_matrix share an SM up to 2176.  From cold caches,
// folded and by row pairs: 2 x 300 on 2 x 300 (1797 offsets, 4 heads) 16 and 34 us, 64 x 40 on 64 x 40 (711) 52 and 104,
// 16 x 16 on 16 x 16 13 both ways; beyond, the fold would still win (2 x 500 on 2 x 500, 2997: 20 and 35; 2 x 650: 26 and 37).
constexpr int kMaxFoldUnits = 2048;

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// out[h][i][j] = offset table of head h at the pair's offset.  The head's n m
// elements are written as one run of 16-byte vectors (ragged ends element by
// element), so rows of any length give full-width stores; a vector finds its
// first pair by one division and walks from there.  Three heads of 576 x 576 (2 MB)
// take 12 us from cold caches, most of it the launch and the offset table.  Bound by
// the instructions of the walk once the matrix is large, a table look-up and a step
// per element: four heads of 4096 x 4096 take 130 us in fp32 (268 MB, 2.1 TB/s) and
// 118 in bf16 (134 MB).
template <typename T>
__global__ void __launch_bounds__(kDenseThreads) bias_dense(BiasDev b, T *out, int n, int m) {
    extern __shared__ __align__(16) float lut[];
    chain_begin();
    constexpr int kVec = 16 / (int)sizeof(T);
    const int h = blockIdx.y, tid = threadIdx.x;
    fill_offsets<false>(b, h, lut, tid, kDenseThreads);
    __syncthreads();
    const unsigned count = (unsigned)n * (unsigned)m;
    T *base = out + (size_t)h * count;
    const unsigned head = min(count, (unsigned)((16u - (unsigned)(reinterpret_cast<uintptr_t>(base) & 15u)) & 15u) /
                                         (unsigned)sizeof(T));
    const unsigned vecs = (count - head) / kVec, tail = head + vecs * kVec;
    auto value = [&](int i, int j) {
        return lut[min(max(off_key(b, j) - off_query(b, i, b.start), 0), b.entries - 1)];
    };
    if (blockIdx.x == 0) {
        for (unsigned f = tid; f < head; f += kDenseThreads) put(base + f, value((int)(f / m), (int)(f % m)));
        for (unsigned f = tail + tid; f < count; f += kDenseThreads) put(base + f, value((int)(f / m), (int)(f % m)));
    }
    for (unsigned v = blockIdx.x * kDenseThreads + tid; v < vecs; v += gridDim.x * kDenseThreads) {
        const unsigned f = head + v * kVec;
        int i = (int)(f / (unsigned)m), j = (int)(f - (unsigned)i * (unsigned)m);
        int oq = off_query(b, i, b.start), ok = off_key(b, j), ck = b.mode == 2 ? j % b.k_cols : 0;
        __align__(16) T x[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            put(x + e, lut[min(max(ok - oq, 0), b.entries - 1)]);
            if (++j == m) {
                j = ck = ok = 0;
                oq = off_query(b, min(++i, n - 1), b.start);
            } else {
                ok += b.step_c;
                if (b.mode == 2 && ++ck == b.k_cols) {
                    ck = 0;
                    ok += b.step_r * b.P - b.step_c * b.k_cols;
                }
            }
        }
        *reinterpret_cast<uint4 *>(base + f) = *reinterpret_cast<const uint4 *>(x);
    }
}

// The table by offset, times log2(e): thread per offset, all heads of it.
__global__ void __launch_bounds__(128) bias_offsets(BiasDev b, float *out) {
    chain_begin();
    const int at = blockIdx.x * 128 + threadIdx.x, h0 = blockIdx.y * 4;
    if (at >= b.entries + 2 * b.pad + 4) return;   // four zeros behind the last
    const bool in = at < b.entries + 2 * b.pad;
    const int e = min(max(at - b.pad, 0), b.entries - 1);
    const float *row = b.table + (size_t)entry_bucket(b, e) * b.heads;
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = in && h0 + u < b.heads ? row[h0 + u] : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (h0 + u < b.heads) out[(size_t)(h0 + u) * b.offsets_pitch + at] = masked_entry(v[u]) * 1.4426950408889634f;
}

// ---------------------------------------------------------------- gradient
// For one pair of rows (rq, rk) of the two grids the q_cols x k_cols block of
// dbias is summed along its diagonals: with u = q_cols - 1 - cq = s q + r
// (s the key step, r < s) and e = ck + q, the pair's column offset is
// s e + r - (q_cols - 1) - start, so a thread that holds (r, e) and walks q
// adds up one offset in a register, and the threads of a warp read
// neighbouring keys of one row.  An item is a chunk of q of one row pair; its
// diagonal sums are folded into the column buckets (each a range of offsets)
// and left as partials; a second kernel adds the partials of each row bucket
// in a fixed order.
struct GradParams {
    BiasDev b;
    int q_rows, q_cols, k_rows, k_cols, step_r, step_c, start_r, start_c;
    int residues, ch, nchunk, etot, ntile, threads;
    int row_buckets, col_buckets;
    long long n, m;
    int parts;     // matrices [heads][n][m] one behind the other, added up
    float *part;   // [heads][q_rows][k_rows][nchunk][ntile][col_buckets]
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float get(const float *p) { return __ldg(p); }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

template <typename T>
__global__ void __launch_bounds__(256) bias_grad_part(const __grid_constant__ GradParams g, const T *dbias) {
    __shared__ float diag[256];
    chain_begin();
    const int t = threadIdx.x, h = blockIdx.z;
    const int tile = blockIdx.x % g.ntile, chunk = blockIdx.x / g.ntile;
    const int rq = blockIdx.y / g.k_rows, rk = blockIdx.y % g.k_rows;
    const int q0 = chunk * g.ch;
    const int flat = tile * g.threads + t;
    const int r = flat / g.etot, e = q0 + flat % g.etot;
    float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
    if (r < g.residues) {
        const int nr = (g.q_cols - 1 - r) / g.step_c + 1;
        int q = max(q0, e - g.k_cols + 1);
        const int q1 = min(min(q0 + g.ch, nr), e + 1);
        // element (q): query column q_cols - 1 - r - s q, key column e - q
        const T *p = dbias + ((long long)h * g.n + (long long)rq * g.q_cols + (g.q_cols - 1 - r - (long long)g.step_c * q)) * g.m +
                     (long long)rk * g.k_cols + (e - q);
        const long long step = -((long long)g.step_c * g.m + 1), matrix = (long long)g.b.heads * g.n * g.m;
        if (g.parts == 1) {
            for (; q + 8 <= q1; q += 8) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = get(p + u * step);
                a0 += v[0] + v[4];
                a1 += v[1] + v[5];
                a2 += v[2] + v[6];
                a3 += v[3] + v[7];
                p += 8 * step;
            }
        }
        for (; q < q1; ++q, p += step) {   // the matrices side by side
            for (int part = 0; part < g.parts; part += 8) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = part + u < g.parts ? get(p + (part + u) * matrix) : 0.f;
                a0 += v[0] + v[4];
                a1 += v[1] + v[5];
                a2 += v[2] + v[6];
                a3 += v[3] + v[7];
            }
        }
    }
    diag[t] = (a0 + a1) + (a2 + a3);
    __syncthreads();
    float *out = g.part + ((((size_t)h * g.q_rows + rq) * g.k_rows + rk) * (g.nchunk * g.ntile) + blockIdx.x) *
                              (size_t)g.col_buckets;
    const int last = g.step_c * (g.k_cols - 1) + g.q_cols - 1;   // offsets run over o = 0 .. last
    const int shift = g.q_cols - 1 + g.start_c, first = tile * g.threads;
    for (int cb = t; cb < g.col_buckets; cb += g.threads) {
        int lo, hi;
        bucket_range(g.b.cols, cb, lo, hi);
        const int o0 = max(lo + shift, 0), o1 = min(hi + shift, last);
        float s = 0.f;
        // of each residue that the tile holds, the run of e whose offsets s e + r are in [o0, o1]
        for (int rr = first / g.etot; rr < g.residues && rr * g.etot < first + g.threads; ++rr) {
            const int row = rr * g.etot - first;
            int e0 = max(0, -row), e1 = min(g.etot, g.threads - row) - 1;
            e0 = max(e0, (o0 <= rr ? 0 : (o0 - rr - 1) / g.step_c + 1) - q0);
            e1 = min(e1, (o1 < rr ? -1 : (o1 - rr) / g.step_c) - q0);
            for (int e = e0; e <= e1; ++e) s += diag[row + e];
        }
        out[cb] = s;
    }
}

// dtable of one row bucket: the partials of its row pairs, `groups` runs of them added side by side.
__global__ void __launch_bounds__(1024) bias_grad_sum(const __grid_constant__ GradParams g, float *dtable, int width,
                                                      int groups) {
    __shared__ float acc_s[1024];
    chain_begin();
    const int rb = blockIdx.x, h = blockIdx.z;
    const int c = threadIdx.x % width, grp = threadIdx.x / width;
    const int cb = blockIdx.y * width + c;
    const int per = g.nchunk * g.ntile;
    int lo, hi;
    bucket_range(g.b.rows, rb, lo, hi);
    float acc = 0.f;
    if (cb < g.col_buckets) {
        const size_t row = (size_t)g.col_buckets;
        // the runs share out the rows of the query grid (four at a time, their first items side by side), or a
        // sequence's items
        const int by_row = g.q_rows > 1, by = by_row ? 1 : groups;
        for (int rq0 = by_row ? grp : 0; rq0 < g.q_rows; rq0 += by_row ? 4 * groups : 1) {
            const float *p[4];
            int items[4];
            float a[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // row offset step_r rk - rq - start_r in [lo, hi]
                const int rq = rq0 + u * groups;
                const long long base = (long long)rq + g.start_r;
                const long long x0 = lo + base, x1 = hi + base;
                const int k0 = x0 <= 0 ? 0 : (int)min((x0 + g.step_r - 1) / g.step_r, (long long)g.k_rows);
                const int k1 = x1 < 0 ? -1 : (int)min(x1 / g.step_r, (long long)g.k_rows - 1);
                items[u] = (u == 0 || by_row) && rq < g.q_rows && k1 >= k0 ? (k1 - k0 + 1) * per : 0;
                p[u] = g.part + (((size_t)h * g.q_rows + rq) * g.k_rows + k0) * per * row + cb;
                const int first = by_row ? 0 : grp;
                a[u] = first < items[u] ? p[u][(size_t)first * row] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll 4
                for (int it = (by_row ? 0 : grp) + by; it < items[u]; it += by) a[u] += p[u][(size_t)it * row];
            }
            acc += (a[0] + a[1]) + (a[2] + a[3]);
        }
    }
    acc_s[threadIdx.x] = acc;
    __syncthreads();
    if (grp == 0 && cb < g.col_buckets) {
        float s = 0.f;
        for (int u = 0; u < groups; ++u) s += acc_s[u * width + c];
        dtable[((size_t)rb * g.col_buckets + cb) * g.b.heads + h] = s;
    }
}

// ------------------------------------------------- gradient, tile by tile
__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 4 bytes global -> shared
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One 128 x 128 tile of one head's matrix (blockIdx.z: part, head): loaded into
// shared memory, then folded; three CTAs per SM, so one folds while the others
// load.  Bound by the instructions of both: a whole tile's fp32 loads are one
// copy and one address step each (with a check and an address for each, 5 us more).
// The 268 MB of a 64 x 64 grid's four heads from cold caches: 61 us, 87 with the sums
// behind it.
constexpr int kFoldThreads = 512;
template <typename T, int VEC>
__global__ void __launch_bounds__(kFoldThreads, 3) fold_matrix(const __grid_constant__ FoldDev f, const T *dbias) {
    extern __shared__ __align__(16) float fold_smem[];
    chain_begin();
    float *tile = fold_smem, *sums = fold_smem + kFoldTile * kFoldPitch;
    const int tid = threadIdx.x, jt = blockIdx.x, it = blockIdx.y;
    const int part = blockIdx.z / f.heads, h = blockIdx.z % f.heads;
    const TileGeom g = fold_geom(f, it, jt);
    // 4 bytes of a row per lane: whole lines per load, and stores that meet no bank twice (two bf16: once more)
    constexpr int kPerRow = kFoldTile / VEC, kRowsAtOnce = kFoldThreads / kPerRow, kLoads = kFoldTile / kRowsAtOnce;
    const int r0 = tid / kPerRow, c = (tid % kPerRow) * VEC;
    struct __align__(sizeof(T) * VEC) Vec { T v[VEC]; };
    const T *src = dbias + (size_t)blockIdx.z * ((size_t)f.n * f.m) + (size_t)(g.q0 + r0) * f.m + g.j0 + c;
    const size_t step = (size_t)kRowsAtOnce * f.m;
    if (sizeof(T) == 4 && g.nq == kFoldTile && g.nk == kFoldTile) {   // straight into shared memory, all of it in flight
        const uint32_t dst = smem_at(tile + r0 * kFoldPitch + c);
#pragma unroll
        for (int e = 0; e < kLoads; ++e, src += step) copy4(dst + e * (kRowsAtOnce * kFoldPitch * 4), src);
        copies_done();
    } else {
        constexpr int kBatch = 16;
        for (int b = 0; b < kLoads; b += kBatch) {
            Vec x[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e, src += step) {
#pragma unroll
                for (int u = 0; u < VEC; ++u) put(&x[e].v[u], 0.f);
                // a vector is whole or absent: m is a multiple of VEC
                if (r0 + (b + e) * kRowsAtOnce < g.nq && c < g.nk) x[e] = *reinterpret_cast<const Vec *>(src);
            }
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                float *t = tile + (r0 + (b + e) * kRowsAtOnce) * kFoldPitch + c;
#pragma unroll
                for (int u = 0; u < VEC; ++u) t[u] = to_float(x[e].v[u]);
            }
        }
    }
    __syncthreads();
    float *out = fold_block(f, part, h, it, jt);
    const bool direct = fold_direct(f, g);
    fold_offsets(f, g, tile, direct ? out : sums, direct ? f.K : g.dc_n, tid, kFoldThreads);
    if (direct) return;
    __syncthreads();
    fold_buckets(f, g, sums, out, tid, kFoldThreads);
}

// dtable of a row bucket.  1024 tiles at a time: a thread works out whether its
// tile meets the bucket and where its block stands, the tiles that do are lined
// up in order, and then `groups` runs of them are added side by side by `width`
// columns of threads.
struct FoldShare {
    int tile, row, rows, cb_lo, cb_n;   // the block, and its rows of this bucket
};
__global__ void __launch_bounds__(1024) fold_sum(const __grid_constant__ FoldDev f, float *dtable, int width, int groups,
                                                 FastDiv div_ktiles) {
    __shared__ float acc_s[1024];
    __shared__ FoldShare list[1024];
    __shared__ int ahead[33];
    chain_begin();
    const int rb = blockIdx.x, h = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = tid % width, grp = tid / width;
    const int cb = blockIdx.y * width + c;
    int lo, hi;
    bucket_range(f.rows, rb, lo, hi);
    lo = max(lo, -kFar / 2) + f.start_r;   // row differences rk - rq of this bucket
    hi = min(hi, kFar / 2) + f.start_r;
    const int tiles = f.qtiles * f.ktiles;
    const size_t block = (size_t)f.nR * f.K;
    float acc = 0.f;
    for (int t0 = 0; t0 < tiles; t0 += 1024) {
        const int tile = t0 + tid;
        FoldShare mine{tile, 0, 0, 0, 0};
        if (tile < tiles) {
            int jt = tile;
            const int it = split(jt, div_ktiles);
            const TileGeom g = fold_geom(f, it, jt);
            const int d0 = max(lo, g.dr_lo), d1 = min(hi, g.dr_lo + g.dr_n - 1);
            mine = FoldShare{tile, d0 - g.dr_lo, d1 - d0 + 1, g.cb_lo, g.cb_n};
        }
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, mine.rows > 0);
        __syncthreads();   // the previous list has been read
        if (lane == 0) ahead[warp + 1] = __popc(votes);
        if (tid == 0) ahead[0] = 0;
        __syncthreads();
        if (warp == 0) {
            int n = ahead[lane + 1];
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, n, m);
                if (lane >= m) n += up;
            }
            ahead[lane + 1] = n;
        }
        __syncthreads();
        if (mine.rows > 0) list[ahead[warp] + __popc(votes & ((1u << lane) - 1u))] = mine;
        __syncthreads();
        const int count = ahead[32];
        for (int part = 0; part < f.parts; ++part) {
            const float *base = f.part + ((size_t)part * f.heads + h) * tiles * block + cb;
            for (int e0 = grp < groups ? grp : count; e0 < count; e0 += 8 * groups) {   // eight tiles' loads in flight
                const float *b[8];
                int rows[8];
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int e = e0 + u * groups;
                    const FoldShare s = list[min(e, count - 1)];
                    rows[u] = e < count && cb >= s.cb_lo && cb < s.cb_lo + s.cb_n ? s.rows : 0;
                    b[u] = base + s.tile * block + (size_t)s.row * f.K - s.cb_lo;
                    v[u] = rows[u] > 0 ? *b[u] : 0.f;
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    for (int d = 1; d < rows[u]; ++d) v[u] += b[u][(size_t)d * f.K];
                acc += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            }
        }
    }
    acc_s[tid] = acc;
    __syncthreads();
    if (grp == 0 && cb < f.col_buckets) {
        float s = 0.f;
        for (int u = 0; u < groups; ++u) s += acc_s[u * width + c];
        dtable[((size_t)rb * f.col_buckets + cb) * f.heads + h] = s;
    }
}

template <typename T, int VEC>
cudaError_t run_fold_vec(const FoldDev &f, const T *dbias, cudaStream_t s) {
    cudaError_t e = allow_smem<fold_matrix<T, VEC>>();
    if (e != cudaSuccess) return e;
    return launch_plain(fold_matrix<T, VEC>, dim3((unsigned)f.ktiles, (unsigned)f.qtiles, (unsigned)(f.heads * f.parts)), kFoldThreads,
                          kFoldTileBytes + f.units * 4, s, f, dbias);
}

template <typename T>
cudaError_t run_fold(const FoldDev &f, const T *dbias, cudaStream_t s) {
    if (sizeof(T) == 2 && f.m % 2 == 0) return run_fold_vec<T, 2>(f, dbias, s);
    return run_fold_vec<T, 1>(f, dbias, s);
}

void grad_plan(const lisa_rel_bias &b, GradParams &g) {
    g.q_rows = b.q_rows; g.q_cols = b.q_cols;
    g.k_rows = b.k_rows; g.k_cols = b.k_cols;
    g.step_r = b.key_step_rows; g.step_c = b.key_step_cols;
    g.start_r = b.start_rows; g.start_c = b.start_cols;
    g.row_buckets = b.rows.buckets; g.col_buckets = b.cols.buckets;
    g.n = (long long)b.q_rows * b.q_cols;
    g.m = (long long)b.k_rows * b.k_cols;
    g.residues = std::min(g.step_c, g.q_cols);
    const int nmax = (g.q_cols - 1) / g.step_c + 1;
    // Many buckets: longer chunks, so fewer partial rows of them.  From cold caches, chunks of 64 and of 256: 33 buckets
    // (4 heads, 4096 x 512, step 8) 23 and 35 us, 513 buckets (8 heads, 2048 x 1024, step 2) 39 and 40, 2049 (4 heads,
    // 4096 x 1024, step 2) 51 and 45, 8193 of the same 84 and 64.
    g.ch = std::min(nmax, g.col_buckets > 512 ? 256 : 64);
    g.nchunk = (nmax + g.ch - 1) / g.ch;
    g.etot = g.k_cols + g.ch - 1;
    const long long flat = (long long)g.residues * g.etot;
    g.threads = (int)std::min<long long>(256, (flat + 31) / 32 * 32);
    g.ntile = (int)((flat + g.threads - 1) / g.threads);
}

}  // namespace

size_t offsets_bytes(const BiasDev &b) {
    return (size_t)b.heads * b.offsets_pitch * sizeof(float);
}

cudaError_t launch_offsets(const BiasDev &b, float *out, cudaStream_t s) {
    return launch_chained(bias_offsets, dim3((unsigned)((b.entries + 2 * b.pad + 4 + 127) / 128), (unsigned)((b.heads + 3) / 4)), 128, 0, s,
                          b, out);
}

cudaError_t launch_bias_dense(const lisa_rel_bias &b, const BiasDev &dev, void *out, int dtype, cudaStream_t s) {
    const int n = b.q_rows * b.q_cols, m = b.k_rows * b.k_cols;
    const size_t esz = dtype == LISA_BF16 ? 2 : 4;
    const size_t vecs = (size_t)n * m * esz / 16 + 1;
    // enough vectors for a CTA to pay for its offset table, at most about eight CTAs per SM
    size_t blocks = (vecs + kDenseThreads * 4 - 1) / (kDenseThreads * 4);
    blocks = std::max<size_t>(1, std::min<size_t>(blocks, (kSms * 8 + dev.heads - 1) / dev.heads));
    const int bytes = dev.entries * (int)sizeof(float);
    const dim3 grid((unsigned)blocks, (unsigned)dev.heads);
    cudaError_t e;
    if (dtype == LISA_BF16) {
        if ((e = allow_smem<bias_dense<__nv_bfloat16>>()) != cudaSuccess) return e;
        return launch_chained(bias_dense<__nv_bfloat16>, grid, kDenseThreads, bytes, s, dev, static_cast<__nv_bfloat16 *>(out),
                              n, m);
    }
    if ((e = allow_smem<bias_dense<float>>()) != cudaSuccess) return e;
    return launch_chained(bias_dense<float>, grid, kDenseThreads, bytes, s, dev, static_cast<float *>(out), n, m);
}

bool fold_plan(const lisa_rel_bias &b, int heads, int parts, FoldDev &f) {
    f = FoldDev{};
    if (b.key_step_rows != 1 || b.key_step_cols != 1) return false;
    BiasDev dev;
    if (bias_dev(&b, heads, dev) != LISA_OK) return false;
    f.n = b.q_rows * b.q_cols;
    f.m = b.k_rows * b.k_cols;
    f.heads = heads;
    f.parts = parts;
    f.qtiles = (f.n + kFoldTile - 1) / kFoldTile;
    f.ktiles = (f.m + kFoldTile - 1) / kFoldTile;
    f.div_q = fast_div(b.q_cols);
    f.div_k = fast_div(b.k_cols);
    f.start_r = b.start_rows;
    f.start_c = b.start_cols;
    f.rows = dev.rows;
    f.cols = dev.cols;
    f.row_buckets = b.rows.buckets;
    f.col_buckets = b.cols.buckets;
    // rows of a grid that 128 of its tokens can touch
    const int qr = std::min(b.q_rows, (kFoldTile - 2) / b.q_cols + 2), kr = std::min(b.k_rows, (kFoldTile - 2) / b.k_cols + 2);
    f.nR = qr + kr - 1;
    // columns that they can span: 128 tokens that cross a row's end, all of the grid's
    const auto span = [](int rows, int cols) { return rows == 1 ? std::min(kFoldTile, cols) : cols; };
    const int width = span(b.q_rows, b.q_cols) + span(b.k_rows, b.k_cols) - 1;
    f.K = dev.cols.log_rule ? b.cols.buckets : std::min(b.cols.buckets, width);
    const long long units = (long long)f.nR * width;
    f.units = (int)std::min<long long>(units, kMaxFoldUnits);
    return units <= kMaxFoldUnits && f.qtiles <= 65535 && (long long)heads * parts <= 65535 && (long long)f.qtiles * f.ktiles < (1 << 30);
}

size_t fold_bytes(const FoldDev &f) {
    return (size_t)f.parts * f.heads * f.qtiles * f.ktiles * f.nR * f.K * sizeof(float);
}

cudaError_t launch_fold_sum(const FoldDev &f, float *dtable, cudaStream_t s) {
    const int width = std::min(256, (f.col_buckets + 31) / 32 * 32), groups = 1024 / width;
    return launch_chained(fold_sum, dim3((unsigned)f.row_buckets, (unsigned)((f.col_buckets + width - 1) / width), (unsigned)f.heads),
                        1024, 0, s, f, dtable, width, groups, fast_div(f.ktiles));
}

size_t bias_grad_bytes(const lisa_rel_bias &b, int heads, int parts) {
    FoldDev f;
    if (fold_plan(b, heads, parts, f)) return fold_bytes(f);
    GradParams g{};
    grad_plan(b, g);
    return (size_t)heads * g.q_rows * g.k_rows * g.nchunk * g.ntile * g.col_buckets * sizeof(float);
}

cudaError_t launch_bias_grad(const lisa_rel_bias &b, const BiasDev &dev, const void *dbias, int parts, int dtype,
                             float *dtable, void *ws, cudaStream_t s) {
    FoldDev f;
    if (fold_plan(b, dev.heads, parts, f)) {
        f.part = static_cast<float *>(ws);
        cudaError_t e = dtype == LISA_BF16 ? run_fold(f, static_cast<const __nv_bfloat16 *>(dbias), s)
                                           : run_fold(f, static_cast<const float *>(dbias), s);
        return e != cudaSuccess ? e : launch_fold_sum(f, dtable, s);
    }
    GradParams g{};
    g.b = dev;
    g.parts = parts;
    grad_plan(b, g);
    g.part = static_cast<float *>(ws);
    dim3 grid((unsigned)(g.nchunk * g.ntile), (unsigned)(g.q_rows * g.k_rows), (unsigned)dev.heads);
    cudaError_t e = dtype == LISA_BF16
                        ? launch_plain(bias_grad_part<__nv_bfloat16>, grid, g.threads, 0, s, g, static_cast<const __nv_bfloat16 *>(dbias))
                        : launch_plain(bias_grad_part<float>, grid, g.threads, 0, s, g, static_cast<const float *>(dbias));
    if (e != cudaSuccess) return e;
    // 1024 threads as `groups` runs of partials by `width` column buckets
    const int width = std::min(256, (g.col_buckets + 31) / 32 * 32), groups = 1024 / width;
    return launch_plain(bias_grad_sum, dim3((unsigned)g.row_buckets, (unsigned)((g.col_buckets + width - 1) / width), (unsigned)dev.heads),
                          width * groups, 0, s, g, dtable, width, groups);
}

}  // namespace attn
}  // namespace lisa
