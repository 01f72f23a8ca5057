"""Cases of the cross-attention and relative-position-bias operators.

Each case is one call (or, for a training step, one forward and its backward)
on inputs like those that the layer meets: queries of one token grid or
sequence against encoder states of another length, with or without a learned
bias by buckets of the relative position, and the bias matrix by itself with
its gradient.

``run`` computes a case in elementary torch operations (``own`` false) or
through this package (``own`` true); ``exact`` computes it in 64 bits, slice by
slice, from the definition.

Positions.  Query token (r, c) of its grid stands at (r, c) + start, key token
(r, c) at step * (r, c); an offset is the key's position minus the query's.
An axis puts an offset x into a bucket by one of two rules:
  exact  clamp(x, -D, D) + D                                  (2 D + 1 buckets)
  log    N buckets, N / 2 to each side (x > 0 the second half), of these
         E = N / 4 hold |x| = 0 .. E-1 one by one and the rest grow
         geometrically: E + floor(log(|x| / E) / log(D / E) * (N / 2 - E)),
         at most N / 2 - 1
The table's row is row_bucket * column_buckets + column_bucket, its column the
query head.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def _attention(name, direction, dtype, B, heads, kv_heads, q_grid, k_grid, d, bias="none", step=1, ragged=False,
               layout="heads"):
    return {"name": name, "op": "attention", "dir": direction, "dtype": dtype, "B": B, "heads": heads,
            "kv_heads": kv_heads, "qr": q_grid[0], "qc": q_grid[1], "kr": k_grid[0], "kc": k_grid[1], "d": d,
            "bias": bias, "step": step, "ragged": ragged, "layout": layout}


def _bias(name, direction, dtype, heads, q_grid, k_grid, rule, step=1):
    return {"name": name, "op": "bias", "dir": direction, "dtype": dtype, "heads": heads, "qr": q_grid[0],
            "qc": q_grid[1], "kr": k_grid[0], "kc": k_grid[1], "bias": rule, "step": step}


def listed():
    return [
        # a 56 x 56 stage whose keys are pooled 8 x 8: few keys, many queries, the bias of every offset pair
        _attention("pooled_56x56_fwd", "fwd", "bf16", 32, 1, 1, (56, 56), (7, 7), 64, "exact", 8),
        _attention("pooled_56x56_train", "train", "bf16", 32, 1, 1, (56, 56), (7, 7), 64, "exact", 8),
        # 14 x 14 queries reading a padded batch of 24 x 24 encoder states, heads interleaved per token
        _attention("ragged_14x14_24x24_train", "train", "bf16", 64, 3, 3, (1, 196), (1, 576), 64, ragged=True,
                   layout="tokens"),
        # a long grid of queries against a pooled one
        _attention("long_256x256_fwd", "fwd", "bf16", 1, 4, 4, (1, 65536), (1, 1024), 64),
        # a full 64 x 64 grid on both sides, trained with its bias: the largest
        _attention("grid_64x64_train", "train", "bf16", 2, 4, 4, (64, 64), (64, 64), 64, "exact", 1),
        # a decoder's sequence on padded encoder states, shared key heads, bucketed offsets
        _attention("sequence_500x1500_train", "train", "bf16", 8, 12, 4, (1, 500), (1, 1500), 64, "log", ragged=True,
                   layout="tokens"),
        # one token, one image: the smallest call
        _attention("token_196", "token", "bf16", 1, 3, 3, (1, 1), (1, 196), 64),
        # one token for each of 64 sequences, each at its own position
        _attention("token_4096_batch", "token", "bf16", 64, 12, 4, (1, 1), (1, 4096), 64, "log", ragged=True),
        # the narrow fp32 layer
        _attention("f32_14x14_train", "train", "f32", 4, 2, 2, (14, 14), (14, 14), 16, "exact", 1),
        # the bias matrix of a 24 x 24 window, read by a layer of the user's own
        _bias("bias_24x24_fwd", "fwd", "bf16", 3, (24, 24), (24, 24), "exact"),
        # the gradient of a full 64 x 64 grid's bias
        _bias("bias_64x64_grad", "grad", "f32", 4, (64, 64), (64, 64), "exact"),
        # the gradient of a sequence's bucketed bias
        _bias("bias_500x1500_grad", "grad", "bf16", 12, (1, 500), (1, 1500), "log"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _draw_grids(rng, most):
    """A grid of queries (sides up to ``most``) and keys pooled by 1, 2, 4 or 8."""
    qr, qc, step = _spread(rng, 2, most), _spread(rng, 2, most), rng.choice((1, 1, 2, 4, 8))
    return (qr, qc), ((qr + step - 1) // step, (qc + step - 1) // step), step


def draw(rng):
    while True:
        what = rng.choice(("fwd", "train", "train", "token", "bias_fwd", "bias_grad"))
        rule = rng.choice(("exact", "log"))
        if what.startswith("bias"):
            if rule == "exact":
                q, k, step = _draw_grids(rng, 64)
            else:
                q, k, step = (1, _spread(rng, 1, 4096)), (1, _spread(rng, 1, 4096)), 1
            case = _bias("", what[5:], rng.choice(("bf16", "f32")), rng.randint(1, 12), q, k, rule, step)
        else:
            dtype, d = rng.choice((("bf16", 64), ("bf16", 64), ("bf16", 64), ("bf16", 32), ("f32", 16), ("f32", 64)))
            kv, group = rng.randint(1, 4), rng.choice((1, 1, 2, 3, 4))
            B = _spread(rng, 1, 64)
            kind, step = rng.choice(("none", "none", "exact", "log")), 1
            if what == "token":
                q, k = (1, 1), (1, _spread(rng, 1, 8192))
                kind = "none" if kind == "exact" else kind
            elif kind == "exact":
                q, k, step = _draw_grids(rng, 64)
            else:
                q, k = (1, _spread(rng, 1, 16384)), (1, _spread(rng, 1, 4096))
            case = _attention("", what, dtype, B, kv * group, kv, q, k, d, kind, step, rng.random() < 0.5,
                              rng.choice(("heads", "tokens")))
        del case["name"]
        w = work(case)
        limit = 3.0e10 if case["op"] == "attention" and case["dtype"] == "bf16" else 4.0e9
        if w["flops"] <= limit and w["bytes"] <= 2.6e8:
            return case


# ------------------------------------------------------------ sizes and work

def _sizes(case):
    return case["qr"] * case["qc"], case["kr"] * case["kc"]


def _rule(case):
    """(rule, buckets, D) of the row and the column axis."""
    if case["bias"] == "log":
        return ("exact", 1, 0), ("log", 32, 128)
    s = case["step"]
    D = [max(q - 1, s * (k - 1)) for q, k in ((case["qr"], case["kr"]), (case["qc"], case["kc"]))]
    return ("exact", 2 * D[0] + 1, D[0]), ("exact", 2 * D[1] + 1, D[1])


def _lengths(case):
    """The batch's numbers of valid keys, evenly spread; a batch of four or more has one without any."""
    B, m = case["B"], case["kr"] * case["kc"]
    if not case["ragged"]:
        return [m] * B
    out = [max(1, round(m * (b + 1) / B)) for b in range(B)]
    if B >= 4:
        out[0] = 0
    return out


def work(case):
    n, m = _sizes(case)
    e = 2 if case["dtype"] == "bf16" else 4
    h = case["heads"]
    table = 0
    if case["bias"] != "none":
        r, c = _rule(case)
        table = r[1] * c[1] * h * 4
    if case["op"] == "bias":
        return {"bytes": h * n * m * e + table, "flops": h * n * m}
    B, kv, d = case["B"], case["kv_heads"], case["d"]
    keys = sum(_lengths(case))
    q_bytes, kv_bytes = B * h * n * d * e, keys * kv * d * e
    flops = 4 * h * n * keys * d
    if case["dir"] == "train":   # reads q, k, v, dout; writes out, dq and the whole of dk, dv
        return {"bytes": 4 * q_bytes + 2 * kv_bytes + 2 * B * m * kv * d * e + 2 * table, "flops": flops * 7 // 2}
    return {"bytes": 2 * q_bytes + 2 * kv_bytes + table, "flops": flops}


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    n, m = _sizes(case)
    s = {"case": dict(case)}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["bias"] != "none":
        r, c = _rule(case)
        s["table"] = 0.5 * normal(r[1] * c[1], case["heads"])
    if case["op"] == "bias":
        if case["dir"] == "grad":
            s["dbias"] = normal(case["heads"], n, m).to(dt)
    else:
        B, h, kv, d = case["B"], case["heads"], case["kv_heads"], case["d"]
        if case["layout"] == "tokens":   # as a projection leaves them: [B, tokens, heads, d], keys beside values
            s["q"] = normal(B, n, h, d).to(dt).transpose(1, 2)
            pair = normal(B, m, 2, kv, d).to(dt)
            s["k"], s["v"] = pair[:, :, 0].transpose(1, 2), pair[:, :, 1].transpose(1, 2)
        else:
            s["q"], s["k"], s["v"] = normal(B, h, n, d).to(dt), normal(B, kv, m, d).to(dt), normal(B, kv, m, d).to(dt)
        if case["dir"] == "train":
            s["dout"] = normal(B, h, n, d).to(dt)
        if case["ragged"]:
            order = torch.randperm(B, generator=g, device="cuda")
            s["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")[order]
        if case["dir"] == "token" and case["bias"] != "none":
            s["starts"] = torch.randint(0, m, (B,), generator=g, device="cuda", dtype=torch.int32)
    if own:
        s["plan"] = _handle(s)
    return s


def _handle(s):
    """The framework's description of the bias, as a module holds it beside its table."""
    case = s["case"]
    if case["bias"] == "none":
        return None
    from hop_stochastic_vision_gb300 import lisa

    def axis(rule):
        return lisa.exact_buckets(rule[2]) if rule[0] == "exact" else lisa.log_buckets(rule[1], rule[2])

    r, c = _rule(case)
    return lisa.RelativeBias(s["table"], (case["qr"], case["qc"]), (case["kr"], case["kc"]), rows=axis(r),
                             cols=axis(c), key_step=(case["step"], case["step"]),
                             query_start=s.get("starts", (0, 0)))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------- the framework's calls

def _run_own(s):
    from hop_stochastic_vision_gb300 import lisa
    case = s["case"]
    plan = s["plan"] if "plan" in s else _handle(s)
    if case["op"] == "bias":
        if case["dir"] == "fwd":
            return lisa.relative_bias(plan, dtype=_DT[case["dtype"]])
        return lisa.relative_bias_backward(plan, s["dbias"])
    if case["dir"] != "train":
        return lisa.cross_attention(s["q"], s["k"], s["v"], kv_lens=s.get("lens"), bias=plan)
    out, lse = lisa.cross_attention(s["q"], s["k"], s["v"], kv_lens=s.get("lens"), bias=plan, return_lse=True)
    grads = lisa.cross_attention_backward(s["q"], s["k"], s["v"], out, lse, s["dout"], kv_lens=s.get("lens"),
                                          bias=plan)
    return (out,) + tuple(grads)


# ------------------------------------------------------------ the plain form

def _axis_buckets(x, rule):
    kind, count, D = rule
    if kind == "exact":
        return x.clamp(-D, D) + D
    half, exact = count // 2, count // 4
    a = x.abs()
    # in 64 bits, nudged up by less than any inexact value's distance to the next border
    far = torch.log(a.clamp(min=1).double() / exact) / math.log(D / exact) * (half - exact) + 1e-11
    far = (exact + far.floor().long()).clamp(max=half - 1)
    return torch.where(x > 0, half, 0) + torch.where(a < exact, a, far)


def _bucket_map(s):
    """Table rows [n, m], or [B, n, m] where each batch entry has its own position."""
    case = s["case"]
    dev = s["table"].device
    r, c = _rule(case)

    def coords(rows, cols):
        i = torch.arange(rows * cols, device=dev)
        return i // cols, i % cols

    qr, qc = coords(case["qr"], case["qc"])
    kr, kc = coords(case["kr"], case["kc"])
    st = case["step"]
    if "starts" in s:
        qr, qc = qr[None, :, None], qc[None, :, None] + s["starts"].long()[:, None, None]
    else:
        qr, qc = qr[:, None], qc[:, None]
    return _axis_buckets(st * kr - qr, r) * c[1] + _axis_buckets(st * kc - qc, c)


def _run_plain(s):
    case = s["case"]
    dt = _DT[case["dtype"]]
    index = _bucket_map(s) if case["bias"] != "none" else None
    if case["op"] == "bias":
        if case["dir"] == "fwd":
            return s["table"].t()[:, index].to(dt)
        return _table_gradient(s["dbias"], index, s["table"].shape[0])
    h, kv, n, m, B = case["heads"], case["kv_heads"], *_sizes(case), case["B"]
    g, d = h // kv, case["d"]
    scale = 1.0 / math.sqrt(d)
    q = s["q"].float().reshape(B, kv, g, n, d)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    score = torch.matmul(q, k.transpose(-1, -2)) * scale
    if index is not None:
        bias = s["table"][index]                                 # [.., n, m, h]
        bias = bias.permute(0, 3, 1, 2) if bias.dim() == 4 else bias.permute(2, 0, 1)[None]
        score += bias.reshape(-1, kv, g, n, m)
    if "lens" in s:
        score.masked_fill_(torch.arange(m, device=q.device) >= s["lens"].view(B, 1, 1, 1, 1), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p, v)
    if case["dir"] != "train":
        return out.reshape(B, h, n, d).to(dt)
    del score
    do = s["dout"].float().reshape(B, kv, g, n, d)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds = p * (ds - (do * out).sum(-1, keepdim=True))
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * scale
    res = (out.reshape(B, h, n, d).to(dt), dq.reshape(B, h, n, d).to(dt), dk.to(dt), dv.to(dt))
    if index is None:
        return res
    return res + (_table_gradient(ds.reshape(B, h, n, m).sum(0), index, s["table"].shape[0]),)


def _table_gradient(dbias, index, rows):
    """Sum of [h, n, m] over the pairs of each bucket: long sums, in 64 bits."""
    out = torch.zeros(rows, dbias.shape[0], dtype=torch.float64, device=dbias.device)
    for head in range(dbias.shape[0]):
        out[:, head].index_add_(0, index.reshape(-1), dbias[head].reshape(-1).double())
    return out.float()


# ------------------------------------------------------- the definition in 64 bits

def _bucket_of(x, rule):
    """One offset's bucket, in whole numbers."""
    kind, count, D = rule
    if kind == "exact":
        return min(max(x, -D), D) + D
    half, exact = count // 2, count // 4
    side, a = (half if x > 0 else 0), abs(x)
    if a < exact:
        return side + a
    b, steps = exact, half - exact
    # bucket exact + t begins where (a / exact) ^ steps >= (D / exact) ^ t
    while b < half - 1 and a ** steps * exact ** (b + 1 - exact) >= D ** (b + 1 - exact) * exact ** steps:
        b += 1
    return side + b


def _exact_index(case, start=0):
    """Table rows [n, m] from a list of every offset's bucket on each axis."""
    st = case["step"]
    parts = []
    for (nq, nk), rule, begin in zip(((case["qr"], case["kr"]), (case["qc"], case["kc"])), _rule(case), (0, start)):
        lo = -(nq - 1) - begin
        of = torch.tensor([_bucket_of(x, rule) for x in range(lo, st * (nk - 1) - begin + 1)])
        off = st * torch.arange(nk).view(1, nk) - torch.arange(nq).view(nq, 1) - begin
        parts.append(of[off - lo])
    rows, cols = parts
    both = rows[:, None, :, None] * _rule(case)[1][1] + cols[None, :, None, :]
    return both.reshape(case["qr"] * case["qc"], case["kr"] * case["kc"]).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    n, m = _sizes(case)
    h = case["heads"]
    table = s["table"].double() if "table" in s else None
    index = _exact_index(case) if table is not None and "starts" not in s else None
    if case["op"] == "bias":
        if case["dir"] == "fwd":
            return torch.stack([table[:, j][index] for j in range(h)])
        grad = torch.zeros_like(table)
        for j in range(h):
            grad[:, j] = torch.bincount(index.view(-1), weights=s["dbias"][j].double().view(-1),
                                        minlength=table.shape[0])
        return grad
    B, group, d = case["B"], h // case["kv_heads"], case["d"]
    lens = s["lens"].tolist() if "lens" in s else [m] * B
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    out = torch.zeros(B, h, n, d, dtype=torch.float64, device="cuda")
    train = case["dir"] == "train"
    if train:
        do, dq, dk, dv = s["dout"].double(), torch.zeros_like(out), torch.zeros(k.shape).to(k), torch.zeros(k.shape).to(k)
        dbias = torch.zeros(h, n, m, dtype=torch.float64, device="cuda") if table is not None else None
    rows = max(1, (1 << 26) // max(m, 1))
    for b in range(B):
        L = lens[b]
        if L == 0:
            continue
        if "starts" in s:
            index = _exact_index(case, int(s["starts"][b]))
        for j in range(h):
            kk, vv = k[b, j // group, :L], v[b, j // group, :L]
            for i in range(0, n, rows):
                part = slice(i, i + rows)
                x = q[b, j, part] @ kk.T / math.sqrt(d)
                if table is not None:
                    x = x + table[:, j][index[part, :L]]
                p = torch.softmax(x, -1)
                out[b, j, part] = p @ vv
                if train:
                    up = do[b, j, part]
                    dv[b, j // group, :L] += p.T @ up
                    dx = up @ vv.T
                    dx = p * (dx - (p * dx).sum(-1, keepdim=True))
                    dq[b, j, part] = dx @ kk / math.sqrt(d)
                    dk[b, j // group, :L] += dx.T @ q[b, j, part] / math.sqrt(d)
                    if table is not None:
                        dbias[j, part, :L] += dx
    if not train:
        return out
    if table is None:
        return out, dq, dk, dv
    grad = torch.zeros_like(table)
    for j in range(h):
        grad[:, j] = torch.bincount(index.view(-1), weights=dbias[j].view(-1), minlength=table.shape[0])
    return out, dq, dk, dv, grad
