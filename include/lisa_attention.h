/*
 * lisa_attention.h -- C ABI of the softmax cross attention and of the learned
 * relative position bias that stand beside the LiSA layer (lisa.h) in a
 * backbone: queries of one token grid or sequence against an encoder's states
 * of another length (pooled keys, a second resolution, another modality).
 *
 * Per batch entry b and query head h, with kv head g = h / (heads / kv_heads):
 *
 *   s_ij  = scale q_i . k_j + bias_h(i, j)        0 <= j < len_b
 *   p_ij  = exp(s_ij - lse_i),  lse_i = log sum_j exp(s_ij)
 *   o_i   = sum_j p_ij v_j
 *
 * and backward, given dO = dL/dO:
 *
 *   dV_j  = sum_i p_ij dO_i              dP_ij = dO_i . v_j
 *   dS_ij = p_ij (dP_ij - sum_j p_ij dP_ij)
 *   dQ_i  = scale sum_j dS_ij k_j        dK_j  = scale sum_i dS_ij q_i
 *   dtable[bucket(i, j)][h] = sum over b and the pairs of the bucket of dS_ij
 *
 * dK and dV of a kv head are summed over the query heads that share it.
 *
 * Conventions (those of lisa.h where it has one):
 *   - dtype LISA_F32 or LISA_BF16 for Q, K, V, O, dO, dQ, dK, dV; fp32 for lse,
 *     the bias table and its gradient.  LISA_F32 is fp32 arithmetic throughout;
 *     LISA_BF16 multiplies bf16 operands (the tensors, and p and dS rounded to
 *     bf16) with fp32 accumulation, except that the bias gradient sums the
 *     unrounded dS.  Softmax statistics and every sum are fp32 or wider, in a
 *     fixed order: the same call gives the same bits.
 *   - d is 16, 32 or 64.  n and m are any lengths from 0 to 2^22, B and heads
 *     at most 65535, with B heads (n / 64 + 1) and B kv_heads (m / 64 + 1) at
 *     most 2^28; what is larger is LISA_ERR_UNSUPPORTED.
 *   - A tensor [B][heads][tokens][d] is given as a pointer and its strides in
 *     elements; the d elements of a token are contiguous.  Pointers and strides
 *     are multiples of 16 bytes.  A batch or head stride of 0 repeats one entry
 *     (inputs only).  Tokens of one head may not overlap, nor any two
 *     elements of an output: each of its strides has to step over the axes of
 *     smaller strides.  Whether an output overlaps something is told by the
 *     extents, from the first to the last element: an output that lies between
 *     an input's heads or tokens without touching them is refused as well.
 *   - kv_lens (device int32 [B], or NULL for m everywhere) says how many keys of
 *     a batch entry are valid; a value outside 0..m counts as the nearer end.
 *     Keys and values behind it are never used, whatever they hold (NaN
 *     included); their dK and dV are written as 0.
 *   - A row without any key that counts (length 0, or only masked scores) has
 *     o = 0, lse = -inf and gives no gradient.
 *   - Scores (and the bias) of any finite size up to 2^126 give the softmax of the
 *     fp32 scores.
 *   - LISA_BF16's backward takes sum_j p_ij dP_ij as dO_i . o_i from the rounded
 *     output where there are more than 128 keys (without a bias for dQ, dK; with
 *     one for dQ), from the unrounded weights otherwise: what is left of dP there
 *     after that sum is good to one rounding of o.
 *   - The backward takes p from fp32 scores and lse, so p is good to about
 *     |lse| 2^-23 relative; a row of |lse| > 2^20, as only masks of large finite
 *     numbers over a whole row bring it about, gives no gradient.
 *   - The library allocates no device memory.  Every argument is checked on the
 *     host before anything is launched.  Calls are asynchronous on `stream`
 *     (make its device current), never synchronise, and can be captured.  A
 *     workspace needs no initialisation and keeps nothing from one call to the
 *     next, but two calls that overlap on the GPU need one each.
 */
#ifndef LISA_ATTENTION_H_
#define LISA_ATTENTION_H_

#include <stddef.h>

#include "lisa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides of a [B][heads][tokens][d] tensor, in elements. */
typedef struct lisa_strides {
    long long batch, head, token;
} lisa_strides;

/* How one axis puts an offset x (key position minus query position) into a bucket. */
typedef enum lisa_bucket_rule {
    LISA_BUCKETS_EXACT = 0, /* clamp(x, -D, D) + D; buckets = 2 D + 1 */
    LISA_BUCKETS_LOG = 1    /* buckets / 2 to each side, x > 0 the second half; of these E = buckets / 4
                               hold |x| = 0 .. E-1 one by one, the rest
                               E + floor(log(|x| / E) / log(D / E) * E), at most buckets / 2 - 1
                               (decided exactly where |x| is a border) */
} lisa_bucket_rule;

typedef struct lisa_axis_rule {
    int rule;          /* lisa_bucket_rule */
    int buckets;       /* EXACT: 2 D + 1; LOG: a multiple of 4, 4..128 */
    int max_distance;  /* D: EXACT 0..8191; LOG buckets / 4 < D <= 8191 */
} lisa_axis_rule;

/*
 * A learned relative position bias.  Queries are the tokens of a q_rows x
 * q_cols grid, keys those of a k_rows x k_cols one (a sequence is a grid of one
 * row), both in row-major order, so n = q_rows q_cols and m = k_rows k_cols.
 * Query (r, c) stands at (start_rows + r, start_cols + c), key (r, c) at
 * (key_step_rows r, key_step_cols c): keys pooled by s have step s.
 *   table   device fp32 [rows.buckets * cols.buckets][heads]; the pair's row is
 *           row_bucket * cols.buckets + column_bucket.  Entries of -inf, and of
 *           -2^120 or less (a type's lowest value), mask a pair in the attention.
 *   starts  device int32 [B], or NULL: a column start of each batch entry that
 *           replaces start_cols (a token of each sequence at its own position).
 *           Sequences only, and forward only (serving): the bias matrix, its
 *           gradient and the attention's backward refuse it.
 * The offsets that the two grids span, padded to a pitch, are held in shared
 * memory: at most LISA_MAX_OFFSETS of them, or LISA_ERR_UNSUPPORTED.  Grids up
 * to 64 x 64 on both sides fit, and so does every sequence (its offsets stop
 * at the rule's max_distance).
 */
typedef struct lisa_rel_bias {
    const float *table;
    int q_rows, q_cols, k_rows, k_cols;
    int key_step_rows, key_step_cols; /* >= 1 */
    int start_rows, start_cols;
    const int *starts;
    lisa_axis_rule rows, cols;
} lisa_rel_bias;

#define LISA_MAX_OFFSETS 16384

/*
 * The bias matrix: out [heads][n][m] (contiguous, dtype), out[h][i][j] =
 * table[bucket(i, j)][h], rounded once.  It, its gradient and the attention's
 * backward with a bias take n m < 2^31 - 65536, q_rows k_rows <= 65535 and
 * heads ceil(n / 128) ceil(m / 128) <= 2^28 (else LISA_ERR_UNSUPPORTED).
 */
lisa_status lisa_relative_bias(const lisa_rel_bias *bias, int heads, void *out, int dtype, void *stream);

/*
 * Its gradient: dtable [rows.buckets * cols.buckets][heads] fp32, written (not
 * accumulated), the sums of dbias [heads][n][m] (contiguous, dtype) over the
 * pairs of each bucket; 0 for a bucket without pairs.  bias->table is not read
 * and may be NULL.  The workspace holds sums of parts of the matrix and no error
 * word: the kernels have no wait that could give up.
 */
size_t lisa_relative_bias_backward_workspace_bytes(const lisa_rel_bias *bias, int heads);
lisa_status lisa_relative_bias_backward(const lisa_rel_bias *bias, int heads, const void *dbias, int dtype,
                                        float *dtable, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Cross attention.  O and lse are written; lse (fp32 [B][heads][n], contiguous)
 * may be NULL.  bias may be NULL.  scale is finite and > 0 (1 / sqrt(d) as a
 * rule).  O and lse may not overlap an input or each other.  The workspace, 16-byte aligned, may be 0
 * bytes (lisa_cross_attention_workspace_bytes says; 0 too for arguments that the
 * call would reject).  Where it is not, it begins with the call's error word
 * (lisa_query_status); a call without one has no wait that could give up.
 */
size_t lisa_cross_attention_workspace_bytes(int B, int heads, int kv_heads, int n, int m, int d,
                                            const lisa_rel_bias *bias, int dtype);
lisa_status lisa_cross_attention(const void *Q, const lisa_strides *q_strides, const void *K,
                                 const lisa_strides *k_strides, const void *V, const lisa_strides *v_strides,
                                 void *O, const lisa_strides *o_strides, float *lse, int B, int heads,
                                 int kv_heads, int n, int m, int d, float scale, const int *kv_lens,
                                 const lisa_rel_bias *bias, int dtype, void *workspace, size_t workspace_bytes,
                                 void *stream);

/*
 * Its backward pass: O and lse as the forward wrote them, dO the upstream
 * gradient; dQ [B][heads][n][d], dK, dV [B][kv_heads][m][d] (contiguous) and,
 * with a bias, dtable are written, never accumulated, and may not overlap each
 * other or an input.  Where K or V repeats an entry (stride 0), dK and dV are
 * those of the repeated tensor, one entry for each repeat.  dtable is NULL
 * exactly when bias is.  The workspace begins with the call's error word.  With a
 * bias it may be large: LISA_F32, and LISA_BF16 where a key step is above 1 or
 * 128 tokens span more than 2048 offsets, hold dS as matrices of heads n m
 * floats, one for each part of the batch that runs side by side (12 heads of
 * 16384 x 4096: 3.2 GB).
 */
size_t lisa_cross_attention_backward_workspace_bytes(int B, int heads, int kv_heads, int n, int m, int d,
                                                     const lisa_rel_bias *bias, int dtype);
lisa_status lisa_cross_attention_backward(const void *Q, const lisa_strides *q_strides, const void *K,
                                          const lisa_strides *k_strides, const void *V,
                                          const lisa_strides *v_strides, const void *O,
                                          const lisa_strides *o_strides, const float *lse, const void *dO,
                                          const lisa_strides *do_strides, void *dQ, void *dK, void *dV,
                                          float *dtable, int B, int heads, int kv_heads, int n, int m, int d,
                                          float scale, const int *kv_lens, const lisa_rel_bias *bias, int dtype,
                                          void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LISA_ATTENTION_H_ */
