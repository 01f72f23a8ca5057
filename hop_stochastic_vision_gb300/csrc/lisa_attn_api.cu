// lisa_attn_api.cu -- the C ABI of the cross attention and the relative
// position bias: argument checks, the bias rule as the kernels read it, the
// workspace carve-up and the dispatch.  Every check runs before the first launch.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "lisa_args.h"
#include "lisa_attention.h"
#include "lisa_attn.h"

namespace lisa {
namespace attn {
namespace {

constexpr int kMaxTokens = 1 << 22;      // queries or keys of one head
constexpr int kMaxGridDim = 65535;       // batch entries and heads
constexpr long long kMaxItems = 1LL << 28;
constexpr int kMaxDistance = 8191;
constexpr long long kMaxPosition = 1LL << 28;

// A sequence's offsets continue at both ends, so that a tile of 128 keys and 32
// queries with any offset inside the table needs no clamping.
constexpr int kOffsetPad = 192;
// Offsets of a head in memory: four zeros behind the last, then up to 256 bytes.
int offsets_pitch(int entries, int pad) { return (entries + 2 * pad + 4 + 63) / 64 * 64; }

lisa_status axis_dev(const lisa_axis_rule &r, AxisDev &a) {
    a = AxisDev{};
    if (r.rule == LISA_BUCKETS_EXACT) {
        if (r.max_distance < 0 || r.buckets != 2 * (long long)r.max_distance + 1) return LISA_ERR_INVALID_ARG;
        if (r.max_distance > kMaxDistance) return LISA_ERR_UNSUPPORTED;
        a.D = r.max_distance;
        return LISA_OK;
    }
    if (r.rule != LISA_BUCKETS_LOG) return LISA_ERR_INVALID_ARG;
    if (r.buckets < 4 || r.buckets % 4 != 0 || r.max_distance <= r.buckets / 4) return LISA_ERR_INVALID_ARG;
    if (r.buckets > 128 || r.max_distance > kMaxDistance) return LISA_ERR_UNSUPPORTED;
    a.log_rule = 1;
    a.half = r.buckets / 2;
    a.nexact = r.buckets / 4;
    a.D = r.max_distance;
    a.nthr = a.half - a.nexact - 1;
    const double E = a.nexact, ratio = (double)a.D / E;
    for (int t = 0; t < a.nthr; ++t) {
        // far bucket t + 1 begins at E ratio^((t + 1) / E); a border that is a
        // whole number is one of its own bucket, whatever pow's last bit says
        const double x = E * std::pow(ratio, (double)(t + 1) / E);
        const double near = std::nearbyint(x);
        a.thr[t] = (int)(std::fabs(x - near) <= 1e-12 * x ? near : std::ceil(x));
    }
    return LISA_OK;
}

}  // namespace

lisa_status bias_dev(const lisa_rel_bias *b, int heads, BiasDev &dev) {
    dev = BiasDev{};
    if (!b || heads < 1) return LISA_ERR_INVALID_ARG;
    if (b->q_rows < 1 || b->q_cols < 1 || b->k_rows < 1 || b->k_cols < 1) return LISA_ERR_INVALID_ARG;
    if (b->key_step_rows < 1 || b->key_step_cols < 1) return LISA_ERR_INVALID_ARG;
    if (heads > kMaxGridDim) return LISA_ERR_UNSUPPORTED;
    if ((long long)b->q_rows * b->q_cols > kMaxTokens || (long long)b->k_rows * b->k_cols > kMaxTokens)
        return LISA_ERR_UNSUPPORTED;
    lisa_status st = axis_dev(b->rows, dev.rows);
    if (st == LISA_OK) st = axis_dev(b->cols, dev.cols);
    if (st != LISA_OK) return st;
    const long long span_r = (long long)b->key_step_rows * (b->k_rows - 1);
    const long long span_c = (long long)b->key_step_cols * (b->k_cols - 1);
    if (span_r > kMaxPosition || span_c > kMaxPosition || std::llabs((long long)b->start_rows) > kMaxPosition ||
        std::llabs((long long)b->start_cols) > kMaxPosition)
        return LISA_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(b->table) & 3u) != 0 || (reinterpret_cast<uintptr_t>(b->starts) & 3u) != 0)
        return LISA_ERR_INVALID_ARG;
    dev.table = b->table;
    dev.heads = heads;
    dev.q_cols = b->q_cols;
    dev.k_cols = b->k_cols;
    dev.step_r = b->key_step_rows;
    dev.step_c = b->key_step_cols;
    dev.start = b->start_cols;
    dev.starts = b->starts;
    dev.col_buckets = b->cols.buckets;
    if (b->q_rows == 1 && b->k_rows == 1) {
        dev.mode = 1;
        dev.lo_r = -b->start_rows;   // the rows' one offset
        const long long D = dev.cols.D;
        long long lo = -D, hi = D;
        if (!b->starts) {
            lo = std::min(std::max(-(long long)(b->q_cols - 1) - b->start_cols, -D), D);
            hi = std::min(std::max(span_c - b->start_cols, -D), D);
        }
        dev.lo_c = (int)lo;
        dev.hi_c = (int)hi;
        dev.entries = (int)(hi - lo + 1);
        dev.pad = kOffsetPad;
        dev.offsets_pitch = offsets_pitch(dev.entries, dev.pad);
        return LISA_OK;
    }
    if (b->starts) return LISA_ERR_INVALID_ARG;
    dev.mode = 2;
    const long long nr = span_r + b->q_rows, nc = span_c + b->q_cols;
    const long long P = nc + ((b->q_cols - nc) % 32 + 32) % 32;
    if (nr * P > LISA_MAX_OFFSETS) return LISA_ERR_UNSUPPORTED;
    dev.P = (int)P;
    dev.div_P = fast_div((int)P);
    dev.div_q = fast_div(b->q_cols);
    dev.div_k = fast_div(b->k_cols);
    dev.run_q = b->q_cols % 4 == 0;
    dev.run_k = b->k_cols % 4 == 0 && b->key_step_cols == 1;
    dev.lo_r = -(b->q_rows - 1) - b->start_rows;
    dev.lo_c = -(b->q_cols - 1) - b->start_cols;
    dev.c0 = (b->q_rows - 1) * dev.P + b->q_cols - 1;
    dev.entries = (int)(nr * P);
    dev.offsets_pitch = offsets_pitch(dev.entries, 0);
    return LISA_OK;
}

namespace {

lisa_status check_sizes(int B, int heads, int kv_heads, int n, int m, int d, int dtype) {
    if (B < 0 || heads < 0 || kv_heads < 0 || n < 0 || m < 0) return LISA_ERR_INVALID_ARG;
    if (dtype != LISA_F32 && dtype != LISA_BF16) return LISA_ERR_INVALID_ARG;
    if (d < 1 || (heads > 0 && (kv_heads < 1 || heads % kv_heads != 0))) return LISA_ERR_INVALID_ARG;
    if (d != 16 && d != 32 && d != 64) return LISA_ERR_UNSUPPORTED;
    if (n > kMaxTokens || m > kMaxTokens || B > kMaxGridDim || heads > kMaxGridDim) return LISA_ERR_UNSUPPORTED;
    // work items of 64 rows or more, shared out by ints
    if ((long long)B * heads * (n / 64 + 1) > kMaxItems || (long long)B * kv_heads * (m / 64 + 1) > kMaxItems)
        return LISA_ERR_UNSUPPORTED;
    return LISA_OK;
}

// Shared by the forward and the backward: everything but the outputs.
lisa_status fill(Problem &p, const void *Q, const lisa_strides *qs, const void *K, const lisa_strides *ks,
                 const void *V, const lisa_strides *vs, int B, int heads, int kv_heads, int n, int m, int d,
                 float scale, const int *kv_lens, const lisa_rel_bias *bias, int dtype) {
    lisa_status st = check_sizes(B, heads, kv_heads, n, m, d, dtype);
    if (st != LISA_OK) return st;
    if (!(scale > 0.f) || !std::isfinite(scale)) return LISA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(kv_lens) & 3u) != 0) return LISA_ERR_INVALID_ARG;
    p.B = B; p.heads = heads; p.kv_heads = kv_heads;
    p.group = heads > 0 ? heads / kv_heads : 1;
    p.n = n; p.m = m; p.d = d;
    p.scale = scale;
    p.kv_lens = kv_lens;
    p.dtype = dtype;
    p.splits = p.q_splits = 1;
    if (B == 0 || heads == 0 || n == 0) return LISA_OK;   // the caller deals with empty problems
    const size_t esz = dtype == LISA_BF16 ? 2 : 4;
    if (!Q || !aligned16(Q) || !good_strides(qs, B, heads, n, d, esz, false)) return LISA_ERR_INVALID_ARG;
    p.Q = {Q, qs->batch, qs->head, qs->token};
    if (m > 0) {
        if (!K || !V || !aligned16(K) || !aligned16(V) || !good_strides(ks, B, kv_heads, m, d, esz, false) ||
            !good_strides(vs, B, kv_heads, m, d, esz, false))
            return LISA_ERR_INVALID_ARG;
        p.K = {K, ks->batch, ks->head, ks->token};
        p.V = {V, vs->batch, vs->head, vs->token};
    }
    if (bias && m > 0) {
        if (!bias->table) return LISA_ERR_INVALID_ARG;
        if ((long long)bias->q_rows * bias->q_cols != n || (long long)bias->k_rows * bias->k_cols != m)
            return LISA_ERR_INVALID_ARG;
        st = bias_dev(bias, heads, p.bias);
        if (st != LISA_OK) return st;
    }
    return LISA_OK;
}

// The forward's path and workspace: CUDA cores for fp32; for bf16 one pass over
// the keys where few rows share a key head, 128-row tiles otherwise.
enum class Path { kNoKeys, kSimt, kToken, kTiles };
struct FwdPlan {
    Path path;
    int splits;
    size_t off_stat, off_o, off_table, total;   // kTiles: the error word is at 0
};

FwdPlan forward_plan(int B, int heads, int group, int n, int m, int d, int dtype, const BiasDev &bias) {
    FwdPlan pl{};
    pl.splits = 1;
    pl.path = m == 0 ? Path::kNoKeys : Path::kSimt;
    if (dtype != LISA_BF16 || m == 0) return pl;
    if (token_applies(heads / group, group, n, bias)) {
        pl.path = Path::kToken;
        return pl;
    }
    pl.path = Path::kTiles;
    pl.splits = tc_forward_splits(B, heads, n, m);
    size_t off = kAlign;
    if (pl.splits > 1) {
        const size_t rows = (size_t)pl.splits * B * heads * n;
        pl.off_stat = off;
        off = align_up(off + rows * sizeof(float2));
        pl.off_o = off;
        off = align_up(off + rows * d * sizeof(float));
    }
    pl.off_table = off;
    if (bias.mode) off = align_up(off + offsets_bytes(bias));
    pl.total = off;
    return pl;
}

struct BwdPlan {
    bool tc;
    int q_splits, b_splits;
    bool folded;
    FoldDev fold;
    size_t off_delta, off_dk, off_dv, off_table, off_dbias, off_grad, total;   // the error word is at 0
};

BwdPlan backward_plan(int B, int heads, int kv_heads, int n, int m, int d, const lisa_rel_bias *bias, int dtype) {
    BwdPlan pl{};
    pl.tc = dtype == LISA_BF16;
    pl.q_splits = pl.b_splits = 1;
    size_t off = kAlign;
    pl.off_delta = off;
    off = align_up(off + (size_t)B * heads * n * sizeof(float));
    if (pl.tc) pl.q_splits = tc_dkdv_splits(B, kv_heads, heads / kv_heads, n, m);
    if (pl.q_splits > 1) {
        const size_t part = (size_t)pl.q_splits * B * kv_heads * m * d * sizeof(float);
        pl.off_dk = off;
        off = align_up(off + part);
        pl.off_dv = off;
        off = align_up(off + part);
    }
    if (bias) {
        pl.b_splits = pl.tc ? tc_dbias_splits(B, heads, n, m) : simt_dbias_splits(B, heads, n, m);
        pl.off_table = off;
        BiasDev dev;
        if (pl.tc && bias_dev(bias, heads, dev) == LISA_OK) off = align_up(off + offsets_bytes(dev));
        pl.folded = pl.tc && fold_plan(*bias, heads, pl.b_splits, pl.fold);
        pl.off_dbias = off;
        if (!pl.folded) off = align_up(off + (size_t)pl.b_splits * heads * n * m * sizeof(float));
        pl.off_grad = off;
        off = align_up(off + (pl.folded ? fold_bytes(pl.fold) : bias_grad_bytes(*bias, heads, pl.b_splits)));
    }
    pl.total = off;
    return pl;
}

size_t table_floats(const lisa_rel_bias &b, int heads) {
    return (size_t)b.rows.buckets * (size_t)b.cols.buckets * (size_t)heads;
}

// Pairs of one head that the bias matrix and its gradient index with 32 bits,
// and tiles of all heads that they share out.
bool matrix_fits(const lisa_rel_bias &b, int heads) {
    const long long n = (long long)b.q_rows * b.q_cols, m = (long long)b.k_rows * b.k_cols;
    return n * m <= (1LL << 31) - 1 - 65536 && (long long)b.q_rows * b.k_rows <= kMaxGridDim &&
           heads * ((n + 127) / 128) * ((m + 127) / 128) <= kMaxItems;
}

}  // namespace
}  // namespace attn
}  // namespace lisa

using namespace lisa::attn;

extern "C" lisa_status lisa_relative_bias(const lisa_rel_bias *bias, int heads, void *out, int dtype, void *stream) {
    if (dtype != LISA_F32 && dtype != LISA_BF16) return LISA_ERR_INVALID_ARG;
    BiasDev dev;
    const lisa_status st = bias_dev(bias, heads, dev);
    if (st != LISA_OK) return st;
    if (!matrix_fits(*bias, heads)) return LISA_ERR_UNSUPPORTED;
    if (!bias->table || !out || bias->starts || !aligned16(out)) return LISA_ERR_INVALID_ARG;
    const size_t bytes = (size_t)heads * bias->q_rows * bias->q_cols * bias->k_rows * bias->k_cols *
                         (dtype == LISA_BF16 ? 2 : 4);
    if (Span(out, bytes).meets(Span(bias->table, table_floats(*bias, heads) * 4))) return LISA_ERR_INVALID_ARG;
    return status_of(launch_bias_dense(*bias, dev, out, dtype, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t lisa_relative_bias_backward_workspace_bytes(const lisa_rel_bias *bias, int heads) {
    BiasDev dev;
    if (bias_dev(bias, heads, dev) != LISA_OK || !matrix_fits(*bias, heads)) return 0;
    return bias_grad_bytes(*bias, heads, 1);
}

extern "C" lisa_status lisa_relative_bias_backward(const lisa_rel_bias *bias, int heads, const void *dbias, int dtype,
                                                   float *dtable, void *workspace, size_t workspace_bytes,
                                                   void *stream) {
    if (dtype != LISA_F32 && dtype != LISA_BF16) return LISA_ERR_INVALID_ARG;
    BiasDev dev;
    const lisa_status st = bias_dev(bias, heads, dev);
    if (st != LISA_OK) return st;
    if (!matrix_fits(*bias, heads)) return LISA_ERR_UNSUPPORTED;
    if (!dbias || !dtable || bias->starts || !aligned16(dbias) || (reinterpret_cast<uintptr_t>(dtable) & 3u) != 0)
        return LISA_ERR_INVALID_ARG;
    const size_t bytes = (size_t)heads * bias->q_rows * bias->q_cols * bias->k_rows * bias->k_cols *
                         (dtype == LISA_BF16 ? 2 : 4);
    if (Span(dtable, table_floats(*bias, heads) * 4).meets(Span(dbias, bytes))) return LISA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < bias_grad_bytes(*bias, heads, 1)) return LISA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return LISA_ERR_INVALID_ARG;
    return status_of(
        launch_bias_grad(*bias, dev, dbias, 1, dtype, dtable, workspace, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t lisa_cross_attention_workspace_bytes(int B, int heads, int kv_heads, int n, int m, int d,
                                                       const lisa_rel_bias *bias, int dtype) {
    if (check_sizes(B, heads, kv_heads, n, m, d, dtype) != LISA_OK || B == 0 || heads == 0 || n == 0) return 0;
    BiasDev dev{};
    if (bias && m > 0 && bias_dev(bias, heads, dev) != LISA_OK) return 0;
    return forward_plan(B, heads, heads / kv_heads, n, m, d, dtype, dev).total;
}

extern "C" lisa_status lisa_cross_attention(const void *Q, const lisa_strides *q_strides, const void *K,
                                            const lisa_strides *k_strides, const void *V,
                                            const lisa_strides *v_strides, void *O, const lisa_strides *o_strides,
                                            float *lse, int B, int heads, int kv_heads, int n, int m, int d,
                                            float scale, const int *kv_lens, const lisa_rel_bias *bias, int dtype,
                                            void *workspace, size_t workspace_bytes, void *stream) {
    Problem p{};
    lisa_status st = fill(p, Q, q_strides, K, k_strides, V, v_strides, B, heads, kv_heads, n, m, d, scale, kv_lens,
                          bias, dtype);
    if (st != LISA_OK) return st;
    if (B == 0 || heads == 0 || n == 0) return LISA_OK;
    const size_t esz = dtype == LISA_BF16 ? 2 : 4;
    if (!O || !aligned16(O) || !good_strides(o_strides, B, heads, n, d, esz, true)) return LISA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return LISA_ERR_INVALID_ARG;
    const Span outs[2] = {Span(O, extent(o_strides, B, heads, n, d, esz)), Span(lse, lse ? (size_t)B * heads * n * 4 : 0)};
    const Span ins[6] = {Span(Q, extent(q_strides, B, heads, n, d, esz)),
                         Span(K, m > 0 ? extent(k_strides, B, kv_heads, m, d, esz) : 0),
                         Span(V, m > 0 ? extent(v_strides, B, kv_heads, m, d, esz) : 0),
                         Span(kv_lens, kv_lens ? (size_t)B * 4 : 0),
                         Span(bias ? bias->table : nullptr, p.bias.mode ? table_floats(*bias, heads) * 4 : 0),
                         Span(p.bias.starts, p.bias.starts ? (size_t)B * 4 : 0)};
    if (outs[0].meets(outs[1])) return LISA_ERR_INVALID_ARG;
    for (const Span &x : outs)
        for (const Span &in : ins)
            if (x.meets(in)) return LISA_ERR_INVALID_ARG;
    p.O = {O, o_strides->batch, o_strides->head, o_strides->token};
    p.lse = lse;
    const FwdPlan pl = forward_plan(B, heads, p.group, n, m, d, dtype, p.bias);
    if (pl.total > 0) {
        if (!workspace || workspace_bytes < pl.total) return LISA_ERR_WORKSPACE;
        if (!aligned16(workspace)) return LISA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (pl.path == Path::kNoKeys) return status_of(launch_no_keys(p, cs));
    if (pl.path == Path::kSimt) return status_of(launch_simt_forward(p, cs));
    if (pl.path == Path::kToken) return status_of(launch_token(p, cs));
    char *ws = static_cast<char *>(workspace);
    p.splits = pl.splits;
    p.stat_part = reinterpret_cast<float2 *>(ws + pl.off_stat);
    p.o_part = reinterpret_cast<float *>(ws + pl.off_o);
    if (p.bias.mode) {
        float *t = reinterpret_cast<float *>(ws + pl.off_table);
        const cudaError_t e = launch_offsets(p.bias, t, cs);
        if (e != cudaSuccess) return LISA_ERR_CUDA;
        p.bias.offsets = t;
    }
    return status_of(launch_tc_forward(p, reinterpret_cast<int *>(ws), cs));
}

extern "C" size_t lisa_cross_attention_backward_workspace_bytes(int B, int heads, int kv_heads, int n, int m, int d,
                                                                const lisa_rel_bias *bias, int dtype) {
    if (check_sizes(B, heads, kv_heads, n, m, d, dtype) != LISA_OK) return 0;
    if (B == 0 || heads == 0 || n == 0 || m == 0) return 0;
    if (bias) {
        BiasDev dev;
        if (bias_dev(bias, heads, dev) != LISA_OK || !matrix_fits(*bias, heads)) return 0;
    }
    return backward_plan(B, heads, kv_heads, n, m, d, bias, dtype).total;
}

extern "C" lisa_status lisa_cross_attention_backward(
    const void *Q, const lisa_strides *q_strides, const void *K, const lisa_strides *k_strides, const void *V,
    const lisa_strides *v_strides, const void *O, const lisa_strides *o_strides, const float *lse, const void *dO,
    const lisa_strides *do_strides, void *dQ, void *dK, void *dV, float *dtable, int B, int heads, int kv_heads, int n,
    int m, int d, float scale, const int *kv_lens, const lisa_rel_bias *bias, int dtype, void *workspace,
    size_t workspace_bytes, void *stream) {
    Problem p{};
    lisa_status st = fill(p, Q, q_strides, K, k_strides, V, v_strides, B, heads, kv_heads, n, m, d, scale, kv_lens,
                          bias, dtype);
    if (st != LISA_OK) return st;
    if ((bias == nullptr) != (dtable == nullptr)) return LISA_ERR_INVALID_ARG;
    if (bias && bias->starts) return LISA_ERR_INVALID_ARG;   // dS is summed over the batch pair by pair
    if ((reinterpret_cast<uintptr_t>(dtable) & 3u) != 0) return LISA_ERR_INVALID_ARG;
    const size_t esz = dtype == LISA_BF16 ? 2 : 4;
    const size_t dq_bytes = (size_t)B * heads * n * d * esz, dk_bytes = (size_t)B * kv_heads * m * d * esz;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool empty = dq_bytes == 0 || dk_bytes == 0;
    if (empty && bias) {   // the table's size has to make sense before it is written
        AxisDev a;
        st = axis_dev(bias->rows, a);
        if (st == LISA_OK) st = axis_dev(bias->cols, a);
        if (st != LISA_OK) return st;
    }
    if ((dq_bytes && !dQ) || (dk_bytes && (!dK || !dV)) || (!empty && (!O || !lse || !dO))) return LISA_ERR_INVALID_ARG;
    if (!aligned16(O) || !aligned16(dO) || !aligned16(dQ) || !aligned16(dK) || !aligned16(dV) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
        return LISA_ERR_INVALID_ARG;
    if (!empty &&
        (!good_strides(o_strides, B, heads, n, d, esz, false) || !good_strides(do_strides, B, heads, n, d, esz, false)))
        return LISA_ERR_INVALID_ARG;
    // an empty problem's inputs need not be there, but where they are they are not written
    const auto span = [&](const void *t, const lisa_strides *s, int h, int tokens) {
        return Span(t, t && s && B > 0 && h > 0 && tokens > 0 ? extent(s, B, h, tokens, d, esz) : 0);
    };
    const Span outs[4] = {Span(dQ, dq_bytes), Span(dK, dk_bytes), Span(dV, dk_bytes),
                          Span(dtable, bias ? table_floats(*bias, heads) * 4 : 0)};
    const Span ins[8] = {span(Q, q_strides, heads, n), span(K, k_strides, kv_heads, m), span(V, v_strides, kv_heads, m),
                         span(O, o_strides, heads, n), span(dO, do_strides, heads, n),
                         Span(lse, lse ? (size_t)B * heads * n * 4 : 0), Span(kv_lens, kv_lens ? (size_t)B * 4 : 0),
                         Span(bias ? bias->table : nullptr, bias && bias->table ? table_floats(*bias, heads) * 4 : 0)};
    for (int a = 0; a < (bias ? 4 : 3); ++a) {
        for (const Span &in : ins)
            if (outs[a].meets(in)) return LISA_ERR_INVALID_ARG;
        for (int c = 0; c < a; ++c)
            if (outs[a].meets(outs[c])) return LISA_ERR_INVALID_ARG;
    }
    if (empty) {   // nothing to differentiate: what there is of the gradients is 0
        if ((dq_bytes && cudaMemsetAsync(dQ, 0, dq_bytes, cs) != cudaSuccess) ||
            (dk_bytes && (cudaMemsetAsync(dK, 0, dk_bytes, cs) != cudaSuccess ||
                          cudaMemsetAsync(dV, 0, dk_bytes, cs) != cudaSuccess)) ||
            (bias && heads > 0 && cudaMemsetAsync(dtable, 0, table_floats(*bias, heads) * 4, cs) != cudaSuccess))
            return LISA_ERR_CUDA;
        return LISA_OK;
    }
    if (bias && !matrix_fits(*bias, heads)) return LISA_ERR_UNSUPPORTED;
    const BwdPlan pl = backward_plan(B, heads, kv_heads, n, m, d, bias, dtype);
    if (!workspace || workspace_bytes < pl.total) return LISA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return LISA_ERR_INVALID_ARG;
    p.O = {O, o_strides->batch, o_strides->head, o_strides->token};
    p.dO = {dO, do_strides->batch, do_strides->head, do_strides->token};
    p.lse = const_cast<float *>(lse);
    p.dQ = dQ;
    p.dK = dK;
    p.dV = dV;
    char *ws = static_cast<char *>(workspace);
    p.err = reinterpret_cast<int *>(ws);
    p.delta = reinterpret_cast<float *>(ws + pl.off_delta);
    p.q_splits = pl.q_splits;
    p.dk_part = reinterpret_cast<float *>(ws + pl.off_dk);
    p.dv_part = reinterpret_cast<float *>(ws + pl.off_dv);
    p.b_splits = pl.b_splits;
    p.dbias = reinterpret_cast<float *>(ws + pl.off_dbias);
    p.folded = pl.folded;
    p.fold = pl.fold;
    p.fold.part = reinterpret_cast<float *>(ws + pl.off_grad);
    cudaError_t e;
    if (pl.tc) {
        e = cudaSuccess;
        if (bias) {
            float *t = reinterpret_cast<float *>(ws + pl.off_table);
            e = launch_offsets(p.bias, t, cs);
            p.bias.offsets = t;
        }
        if (e == cudaSuccess) e = launch_tc_backward(p, reinterpret_cast<int *>(ws), cs);
    } else {
        e = launch_simt_dq(p, cs);
        if (e == cudaSuccess) e = launch_simt_dkdv(p, cs);
        if (e == cudaSuccess && bias) e = launch_simt_dbias(p, cs);
    }
    // the tiles' bucket sums of the batch's dS, or its matrix and then as the bias matrix's own gradient
    if (e == cudaSuccess && bias && pl.folded)
        e = launch_fold_sum(p.fold, dtable, cs);
    else if (e == cudaSuccess && bias)
        e = launch_bias_grad(*bias, p.bias, p.dbias, pl.b_splits, LISA_F32, dtable, ws + pl.off_grad, cs);
    return status_of(e);
}
