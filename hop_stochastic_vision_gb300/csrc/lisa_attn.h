// lisa_attn.h -- host-side problem description of the cross attention and the
// relative position bias, the device view of the bias rule, and the launcher
// entry points of the kernels.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "lisa_attention.h"

namespace lisa {
namespace attn {

// The plans share work out over GB300's SMs without asking the device: a workspace's size is
// known before there is one.
constexpr int kSms = 152;

// Division by a number fixed for the launch: n / d = (umulhi(mul, n) + n) >> shift
// for 0 <= n < 2^31 (the round-up method for 32-bit dividends, one bit to spare).
struct FastDiv {
    unsigned d, mul, shift;
};
inline FastDiv fast_div(int d) {
    FastDiv f{(unsigned)d, 0, 0};
    while ((1ULL << f.shift) < (unsigned long long)d) ++f.shift;
    f.mul = (unsigned)((((1ULL << f.shift) - (unsigned long long)d) << 32) / (unsigned long long)d + 1);
    return f;
}

// One axis of the bucket rule as the kernels read it.  The log rule's borders
// are whole numbers found on the host: thr[t] is the smallest |x| of far
// bucket t + 1 (buckets E + 1, E + 2, ...), so no kernel takes a logarithm.
struct AxisDev {
    int log_rule;      // 0: exact
    int half, nexact;  // log: buckets per side, of these one by one
    int D;
    int nthr;
    int thr[32];
};

// The bias as the kernels read it.  Pair (i, j) has the offset index
//   sequence  clamp(step_c j - i - start, lo_c, hi_c) - lo_c
//   grid      a(j) - b(i) + c0, a(j) = step_r P rk + step_c ck, b(i) = P rq + cq
// into a table of `entries` values, one per offset, that each CTA gathers from
// the bucket table for its head.  The pitch P is at least the number of column
// offsets and congruent to q_cols modulo 32: 32 consecutive queries of one key
// then fall into 32 different shared-memory banks, across row ends too.
struct BiasDev {
    int mode;          // 0 none, 1 sequence, 2 grid
    int entries;
    const float *table;
    const float *offsets;   // tensor-core kernels: [heads][offsets_pitch], the table by offset, times log2(e)
    int offsets_pitch;
    int pad;                // sequence: the outermost values repeated so often at either end
    int heads;
    int q_cols, k_cols, P, step_r, step_c, c0;
    FastDiv div_q, div_k, div_P;   // by q_cols, k_cols, P
    int start;         // sequence: column start
    const int *starts; // sequence: per batch entry
    int lo_r, lo_c, hi_c;
    int run_q, run_k;  // grid: four queries, keys from a multiple of four have consecutive offsets
    int col_buckets;
    AxisDev rows, cols;
};

// Sums of pairs over the buckets, tile by tile (lisa_fold.cuh).
struct FoldDev {
    int n, m, heads, qtiles, ktiles, parts;   // parts: sums to add up per tile (splits of the batch)
    FastDiv div_q, div_k;                      // by the grids' columns
    int start_r, start_c;
    AxisDev rows, cols;
    int row_buckets, col_buckets;
    int nR, K;         // a tile's block: at most nR row differences, K column buckets
    int units;         // at most so many offsets in a tile
    float *part;       // [parts][heads][qtiles][ktiles][nR][K]
};

struct Tensor {
    const void *p;
    long long sb, sh, st;  // strides in elements
};

struct Problem {
    Tensor Q, K, V, O, dO;
    float *lse;
    int B, heads, kv_heads, group, n, m, d;
    float scale;
    const int *kv_lens;
    int dtype;
    BiasDev bias;
    void *dQ, *dK, *dV;
    int *err;              // fp32 backward: the workspace's error word, cleared
    float *delta;          // [B][heads][n]: sum_j p dP, written by the dQ kernel
    // dS summed over (parts of) the batch: folded tile by tile, or as matrices
    int folded;
    FoldDev fold;
    float *dbias;          // not folded: [b_splits][heads][n][m] fp32
    int b_splits;
    // forward split over the keys
    int splits;
    float *o_part;         // [splits][B][heads][n][d], each over its own sum
    float2 *stat_part;     // [splits][B][heads][n]: reference (in units of log 2), sum
    // dK / dV split over the queries
    int q_splits;
    float *dk_part, *dv_part;  // [q_splits][B][kv_heads][m][d]
};

// --- plans -------------------------------------------------------------------
// Fills `dev` from the public struct; checks everything but the batch.
lisa_status bias_dev(const lisa_rel_bias *b, int heads, BiasDev &dev);

// --- launchers ---------------------------------------------------------------
cudaError_t launch_bias_dense(const lisa_rel_bias &b, const BiasDev &dev, void *out, int dtype, cudaStream_t s);
// How the bucket sums of `parts` matrices are taken: tile by tile where the
// grids have the same spacing, from the matrices otherwise.
bool fold_plan(const lisa_rel_bias &b, int heads, int parts, FoldDev &f);
size_t fold_bytes(const FoldDev &f);
// Adds the tiles' blocks up into dtable.
cudaError_t launch_fold_sum(const FoldDev &f, float *dtable, cudaStream_t s);
size_t bias_grad_bytes(const lisa_rel_bias &b, int heads, int parts);
// Bucket sums of `parts` matrices [heads][n][m], one behind the other, added up.
cudaError_t launch_bias_grad(const lisa_rel_bias &b, const BiasDev &dev, const void *dbias, int parts, int dtype,
                             float *dtable, void *ws, cudaStream_t s);

cudaError_t launch_no_keys(const Problem &p, cudaStream_t s);   // m = 0
cudaError_t launch_simt_forward(const Problem &p, cudaStream_t s);
cudaError_t launch_simt_dq(const Problem &p, cudaStream_t s);
cudaError_t launch_simt_dkdv(const Problem &p, cudaStream_t s);
int simt_dbias_splits(int B, int heads, int n, int m);
cudaError_t launch_simt_dbias(const Problem &p, cudaStream_t s);

// The table by offset, times log2(e), into bias.offsets.
size_t offsets_bytes(const BiasDev &b);
cudaError_t launch_offsets(const BiasDev &b, float *out, cudaStream_t s);

// bf16, a few query rows per key head: one pass over the keys
bool token_applies(int kv_heads, int group, int n, const BiasDev &bias);
cudaError_t launch_token(const Problem &p, cudaStream_t s);

// bf16 on the tensor cores; `err` is the error word of the call's workspace
int tc_forward_splits(int B, int heads, int n, int m);
cudaError_t launch_tc_forward(const Problem &p, int *err, cudaStream_t s);
int tc_dkdv_splits(int B, int kv_heads, int group, int n, int m);
int tc_dbias_splits(int B, int heads, int n, int m);
cudaError_t launch_tc_backward(const Problem &p, int *err, cudaStream_t s);

}  // namespace attn
}  // namespace lisa
