"""Cases of the operators around a prompt: rotary positions, attention over
packed prompts, and a key/value cache held in 4 bits.

Each case is one call, a training step (a forward and its backward), or a store
into the cache and the values read back from it, on inputs like those that a
model which reads images, video or text as a prompt meets.

``run`` computes a case in elementary torch operations (``own`` false) or
through this package (``own`` true); ``exact`` computes it in 64 bits from the
definition.

Rotary positions.  The first 2 P of a token's d elements are P pairs, (p, P + p)
or (2 p, 2 p + 1); pair p belongs to an axis a and turns by the angle
position[a] * frequency[p]:  (x, y) -> (x cos - y sin, x sin + y cos).  Pair i of
the s pairs of an axis has the frequency base ^ (-i / s).  The backward pass
turns the gradients by the opposite angle.

Packed prompts.  Sequences stand one behind the other along the tokens; a query
reads the keys of its own sequence, with ``causal`` those up to itself.

The cache in 4 bits.  A token's 32 neighbouring elements of one key head share
scale = bf16(max |x| / 7); each is held as the whole number x / scale, ties to
even.  Tokens stand in pages of 64 that a table gives to the sequences.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_PAGE = 64      # tokens of a page of the cache
_BASE = 10000.0


# ---------------------------------------------------------------- the cases

def _rotary(name, direction, dtype, B, heads, kv_heads, grid, sections, d, pairing="halves", layout="heads", far=0):
    """``grid`` tokens along (time, height, width); ``sections`` pairs of each of the last axes; ``far`` > 0: single
    tokens anywhere up to there."""
    return {"name": name, "op": "rotary", "dir": direction, "dtype": dtype, "B": B, "heads": heads,
            "kv_heads": kv_heads, "t": grid[0], "r": grid[1], "c": grid[2], "sections": sections, "d": d,
            "pairing": pairing, "layout": layout, "far": far}


def _prompt(name, direction, dtype, lengths, heads, kv_heads, d, causal=True, layout="tokens"):
    return {"name": name, "op": "prompt", "dir": direction, "dtype": dtype,
            "lengths": " ".join(str(x) for x in lengths), "heads": heads, "kv_heads": kv_heads, "d": d,
            "causal": causal, "layout": layout}


def _store(name, dtype, B, n, kv_heads, d, start=0, layout="tokens"):
    return {"name": name, "op": "store", "dtype": dtype, "B": B, "n": n, "kv_heads": kv_heads, "d": d, "start": start,
            "layout": layout}


def _token(name, B, heads, kv_heads, m, d, n=1, ragged=False):
    return {"name": name, "op": "token", "dtype": "bf16", "B": B, "heads": heads, "kv_heads": kv_heads, "m": m, "d": d,
            "n": n, "ragged": ragged}


def listed():
    return [
        # the queries and keys of a 56 x 56 stage by row and column
        _rotary("rotary_56x56_fwd", "fwd", "bf16", 32, 1, 1, (1, 56, 56), "16 16", 64),
        # gradients of a short video's queries and keys by time, row and column, heads interleaved per token
        _rotary("rotary_video_bwd", "bwd", "bf16", 2, 12, 4, (8, 24, 24), "8 12 12", 64, "neighbours", "tokens"),
        # one new token of each of 64 sequences, far out
        _rotary("rotary_token_batch", "fwd", "bf16", 64, 12, 4, (1, 1, 1), "8 12 12", 64, layout="tokens", far=1 << 20),
        # one prompt of 4096 tokens when serving
        _prompt("prompt_4096_fwd", "fwd", "bf16", [4096], 12, 4, 64),
        # a training batch packed from sequences of any length, one of them empty
        _prompt("prompt_packed_train", "train", "bf16",
                [1500, 37, 2048, 1, 700, 0, 4096, 129, 333, 1023, 2500, 64, 1777, 511, 900, 765], 12, 4, 64),
        # images of several resolutions packed into one batch, every patch reads every other
        _prompt("images_packed_train", "train", "bf16", [3136, 196, 784, 576, 196, 1369, 49, 576, 3136, 256, 196, 441],
                3, 3, 64, causal=False),
        # one long prompt, trained: the largest
        _prompt("prompt_16384_train", "train", "bf16", [16384], 4, 4, 64),
        # the narrow fp32 layer
        _prompt("f32_packed_train", "train", "f32", [196, 1, 49, 0, 130], 2, 2, 16, layout="heads"),
        # a padded batch of prompts into the cache
        _store("cache_prompts_8x1500", "bf16", 8, 1500, 4, 64),
        # one new token of each of 64 sequences into the cache
        _store("cache_token_batch", "bf16", 64, 1, 4, 64, start=4000),
        # one token for each of 64 sequences of up to 4096 tokens
        _token("cache_attention_4096_batch", 64, 12, 4, 4096, 64, ragged=True),
        # one token, one image: the smallest call
        _token("cache_attention_196", 1, 3, 3, 196, 64),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _draw_sections(rng, d, axes):
    """Pairs of each axis, at least one, at most d / 2 in all; often all of them."""
    total = d // 2 if rng.random() < 0.7 else rng.randint(axes, d // 2)
    cuts = sorted(rng.sample(range(1, total), axes - 1))
    return " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    while True:
        what = rng.choice(("rotary", "rotary", "prompt", "prompt", "prompt", "store", "token", "token"))
        kv, group = rng.randint(1, 4), rng.choice((1, 1, 2, 3, 4))
        dtype, d = rng.choice((("bf16", 64), ("bf16", 64), ("bf16", 64), ("bf16", 32), ("f32", 16), ("f32", 64)))
        layout = rng.choice(("heads", "tokens"))
        if what == "rotary":
            axes = rng.randint(1, 3)
            grid = [1] * (3 - axes) + [_spread(rng, 1, 64 if axes > 1 else 16384) for _ in range(axes)]
            single = rng.random() < 0.2
            case = _rotary("", rng.choice(("fwd", "bwd")), dtype, _spread(rng, 1, 64), kv * group, kv,
                           (1, 1, 1) if single else grid, _draw_sections(rng, d, axes), d,
                           rng.choice(("halves", "neighbours")), layout, _spread(rng, 64, 1 << 22) if single else 0)
        elif what == "prompt":
            count, most = _spread(rng, 1, 40), _spread(rng, 1, 16384)
            lengths = [rng.choice((0, 1, _spread(rng, 1, most), _spread(rng, 1, most), most)) for _ in range(count)]
            case = _prompt("", rng.choice(("fwd", "train", "train")), dtype, lengths, kv * group, kv, d,
                           rng.random() < 0.7, layout)
        elif what == "store":
            case = _store("", dtype, _spread(rng, 1, 64), _spread(rng, 1, 8192), kv, 64 if d == 64 else 32,
                          rng.choice((0, 0, rng.randint(1, 5000))), layout)
        else:
            case = _token("", _spread(rng, 1, 64), kv * group, kv, _spread(rng, 1, 16384), 64 if d == 64 else 32,
                          rng.choice((1, 1, 1, 2, 4)), rng.random() < 0.5)
        del case["name"]
        w = work(case)
        limit = 4.0e9 if case["op"] == "prompt" and dtype == "f32" else 4.8e11
        if 0 < w["flops"] <= limit and w["bytes"] <= 2.0e8:
            return case


# ------------------------------------------------------------ sizes and work

def _sections(case):
    return [int(x) for x in case["sections"].split()]


def _prompt_lengths(case):
    return [int(x) for x in case["lengths"].split()]


def _cache_lengths(case):
    """Tokens of each sequence, evenly spread where the batch is ragged; a batch of four or more has one without any."""
    B, m = case["B"], case["m"]
    if not case["ragged"]:
        return [m] * B
    out = [max(1, round(m * (b + 1) / B)) for b in range(B)]
    if B >= 4:
        out[0] = 0
    return out


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d, kv = case["d"], case["kv_heads"]
    held = d // 2 + d // 32 * 2                # bytes of a token's key (or value) of one head in the cache
    if case["op"] == "rotary":
        n, axes = case["B"] * case["t"] * case["r"] * case["c"], len(_sections(case))
        values = n * (case["heads"] + kv) * d
        shared = case["far"] == 0              # the batch's tokens stand at the same places
        return {"bytes": 2 * values * e + 4 * axes * (n // case["B"] if shared else n), "flops": 3 * values}
    if case["op"] == "prompt":
        lengths, h = _prompt_lengths(case), case["heads"]
        pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in lengths)
        q_bytes, kv_bytes = sum(lengths) * h * d * e, sum(lengths) * kv * d * e
        if case["dir"] == "train":             # reads q, k, v, dout; writes out, dq, dk, dv
            return {"bytes": 4 * q_bytes + 4 * kv_bytes, "flops": 14 * h * pairs * d}
        return {"bytes": 2 * q_bytes + 2 * kv_bytes, "flops": 4 * h * pairs * d}
    if case["op"] == "store":                  # k, v in; held; out again
        tokens = case["B"] * case["n"] * kv
        return {"bytes": tokens * (4 * d * e + 4 * held), "flops": 4 * tokens * d}
    rows, keys = case["B"] * case["n"] * case["heads"], sum(_cache_lengths(case))
    return {"bytes": keys * kv * 2 * held + 2 * rows * d * e, "flops": 4 * case["n"] * case["heads"] * keys * d}


# ------------------------------------------------------------------- inputs

def _view(g, case, shape, layout):
    """[.., heads, tokens, d] of the case's type, in memory so or as a projection leaves it: heads inside tokens."""
    if layout == "tokens":
        shape = shape[:-3] + (shape[-2], shape[-3], shape[-1])
        return torch.randn(*shape, generator=g, device="cuda").to(_DT[case["dtype"]]).transpose(-3, -2)
    return torch.randn(*shape, generator=g, device="cuda").to(_DT[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": dict(case)}
    d, kv = case["d"], case["kv_heads"]
    if case["op"] == "rotary":
        B, axes = case["B"], len(_sections(case))
        n = case["t"] * case["r"] * case["c"]
        s["q"] = _view(g, case, (B, case["heads"], n, d), case["layout"])
        s["k"] = _view(g, case, (B, kv, n, d), case["layout"])
        if case["far"]:
            s["positions"] = torch.randint(0, case["far"], (axes, B, n), generator=g, device="cuda", dtype=torch.int32)
        else:
            i = torch.arange(n, device="cuda", dtype=torch.int32)
            place = (i // (case["r"] * case["c"]), i // case["c"] % case["r"], i % case["c"])
            s["positions"] = torch.stack(place[3 - axes:])
        if own:
            s["plan"] = _axes(case)
    elif case["op"] == "prompt":
        T = sum(_prompt_lengths(case))
        s["q"] = _view(g, case, (case["heads"], T, d), case["layout"])
        s["k"], s["v"] = (_view(g, case, (kv, T, d), case["layout"]) for _ in range(2))
        if case["dir"] == "train":
            s["dout"] = _view(g, case, (case["heads"], T, d), case["layout"])
        if own:
            s["plan"] = _packed(case)
    else:
        B = case["B"]
        if case["op"] == "store":
            s["k"], s["v"] = (_view(g, case, (B, kv, case["n"], d), case["layout"]) for _ in range(2))
            longest = case["start"] + case["n"]
            s["positions"] = torch.arange(case["start"], longest, device="cuda", dtype=torch.int32).repeat(B, 1)
            lengths = [longest] * B
        else:
            lengths, longest = _cache_lengths(case), case["m"]
            s["q"] = _view(g, case, (B, case["heads"], case["n"], d), "heads")
            k, v = (_view(g, case, (B, kv, longest, d), "heads") for _ in range(2))
            s["codes_k"], s["scales_k"] = _held(k.float())
            s["codes_v"], s["scales_v"] = _held(v.float())
            s["lens"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        # every sequence's pages, anywhere in the pool
        width = max(1, -(-longest // _PAGE))
        used = [-(-x // _PAGE) for x in lengths]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        at = torch.tensor(used, device="cuda").cumsum(0) - torch.tensor(used, device="cuda")
        column = torch.arange(width, device="cuda")
        table = order[(at[:, None] + column).clamp(max=pages - 1)]
        s["table"] = torch.where(column < torch.tensor(used, device="cuda")[:, None], table, -1).to(torch.int32)
        s["pages"] = pages
        if own:
            s["cache"] = _cache(s)
            if case["op"] == "token":
                _fill(s, k, v)
    return s


def _axes(case):
    from hop_stochastic_vision_gb300 import lisa
    return lisa.RotaryAxes(case["d"], _sections(case), base=_BASE, pairing=case["pairing"])


def _packed(case):
    from hop_stochastic_vision_gb300 import lisa
    return lisa.PackedSequences(_prompt_lengths(case), case["heads"], case["kv_heads"], causal=case["causal"])


def _cache(s):
    from hop_stochastic_vision_gb300 import lisa
    return lisa.Cache4(s["pages"], s["case"]["kv_heads"], s["case"]["d"])


def _fill(s, k, v):
    """What the steps before this one have left in the cache."""
    from hop_stochastic_vision_gb300 import lisa
    at = torch.arange(k.shape[2], device="cuda", dtype=torch.int32).repeat(k.shape[0], 1)
    lisa.cache_store(s["cache"], k, v, s["table"], torch.where(at < s["lens"][:, None], at, -1))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------- the framework's calls

def _run_own(s):
    from hop_stochastic_vision_gb300 import lisa
    case = s["case"]
    if case["op"] == "rotary":
        call = lisa.rotary if case["dir"] == "fwd" else lisa.rotary_backward
        return call(s["q"], s["k"], s["positions"], s["plan"])
    if case["op"] == "prompt":
        if case["dir"] != "train":
            return lisa.prompt_attention(s["q"], s["k"], s["v"], s["plan"])
        out, lse = lisa.prompt_attention(s["q"], s["k"], s["v"], s["plan"], return_lse=True)
        return (out,) + tuple(lisa.prompt_attention_backward(s["q"], s["k"], s["v"], out, lse, s["dout"], s["plan"]))
    if case["op"] == "store":
        lisa.cache_store(s["cache"], s["k"], s["v"], s["table"], s["positions"])
        return lisa.cache_read(s["cache"], s["table"], s["positions"], dtype=_DT[case["dtype"]])
    return lisa.cache_attention(s["q"], s["cache"], s["table"], s["lens"])


# ------------------------------------------------------------ the plain form

def _run_plain(s):
    case = s["case"]
    dt = _DT[case["dtype"]]
    if case["op"] == "rotary":
        cos, sin = _turns(s)
        return _turn(s["q"], cos, sin, case["pairing"]).to(dt), _turn(s["k"], cos, sin, case["pairing"]).to(dt)
    if case["op"] == "prompt":
        return _prompt_plain(s, dt)
    if case["op"] == "store":
        return tuple(_stands_for(*_held(s[x].float())).to(dt) for x in ("k", "v"))
    return _token_plain(s, dt)


def _turns(s):
    """Cosines and sines [.., n, P] of the tokens' pairs; far positions need the angle in 64 bits."""
    case = s["case"]
    pos, out = s["positions"], []
    for axis, count in enumerate(_sections(case)):
        i = torch.arange(count, device=pos.device, dtype=torch.float64)
        out.append(pos[axis].double()[..., None] * torch.pow(_BASE, -i / count))
    angle = torch.cat(out, -1)
    if angle.dim() == 3:      # each batch entry its own
        angle = angle[:, None]
    if case["dir"] == "bwd":
        angle = -angle
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, cos, sin, pairing):
    P = cos.shape[-1]
    x = x.float()
    if pairing == "halves":
        a, b, rest = x[..., :P], x[..., P:2 * P], x[..., 2 * P:]
        return torch.cat((a * cos - b * sin, a * sin + b * cos, rest), -1)
    a, b, rest = x[..., 0:2 * P:2], x[..., 1:2 * P:2], x[..., 2 * P:]
    pairs = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((pairs, rest), -1)


def _prompt_plain(s, dt):
    case = s["case"]
    h, kv, d, train = case["heads"], case["kv_heads"], case["d"], case["dir"] == "train"
    g, T, scale = h // kv, s["q"].shape[1], 1.0 / math.sqrt(case["d"])
    out = torch.zeros(h, T, d, dtype=dt, device=s["q"].device)
    if train:
        dq, (dk, dv) = torch.zeros_like(out), (torch.zeros(kv, T, d, dtype=dt, device=out.device) for _ in range(2))
    at = 0
    for L in _prompt_lengths(case):
        rows, at = slice(at, at + L), at + L
        if L == 0:
            continue
        later = torch.ones(L, L, dtype=torch.bool, device=out.device).triu(1) if case["causal"] else None
        step = max(1, (1 << 28) // (g * L * L))               # key heads at once
        for j in range(0, kv, step):
            some = slice(j, min(kv, j + step))
            mine = slice(some.start * g, some.stop * g)
            c = some.stop - some.start
            q = s["q"][mine, rows].float().reshape(c, g, L, d)
            k, v = s["k"][some, rows].float()[:, None], s["v"][some, rows].float()[:, None]
            p = torch.matmul(q, k.transpose(-1, -2)) * scale
            if later is not None:
                p.masked_fill_(later, -math.inf)
            p = torch.exp(p - p.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            o = torch.matmul(p, v)
            out[mine, rows] = o.reshape(c * g, L, d).to(dt)
            if train:
                do = s["dout"][mine, rows].float().reshape(c, g, L, d)
                dv[some, rows] = torch.matmul(p.transpose(-1, -2), do).sum(1).to(dt)
                ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
                dq[mine, rows] = (torch.matmul(ds, k) * scale).reshape(c * g, L, d).to(dt)
                dk[some, rows] = (torch.matmul(ds.transpose(-1, -2), q).sum(1) * scale).to(dt)
    return (out, dq, dk, dv) if train else out


def _held(x):
    """Whole numbers [.., d] and scales [.., d / 32] of fp32 values."""
    groups = x.unflatten(-1, (-1, 32))
    scales = (groups.abs().amax(-1) / 7).to(torch.bfloat16).float()
    codes = torch.round(groups / torch.where(scales == 0, 1.0, scales)[..., None])
    return torch.where(scales[..., None] == 0, 0.0, codes).flatten(-2).to(torch.int8), scales


def _stands_for(codes, scales):
    return codes.float() * scales.repeat_interleave(32, -1)


def _token_plain(s, dt):
    case = s["case"]
    B, h, kv, n, m, d = (case[x] for x in ("B", "heads", "kv_heads", "n", "m", "d"))
    k, v = _stands_for(s["codes_k"], s["scales_k"])[:, :, None], _stands_for(s["codes_v"], s["scales_v"])[:, :, None]
    q = s["q"].float().reshape(B, kv, h // kv, n, d)
    score = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    # the rows are the newest n tokens: each sees the keys up to itself
    i = torch.arange(n, device=q.device)
    sees = s["lens"].view(B, 1) - (n - 1 - i)
    score.masked_fill_(torch.arange(m, device=q.device) >= sees.view(B, 1, 1, n, 1), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p / torch.where(total == 0, 1.0, total), v)
    return out.reshape(B, h, n, d).to(dt)


# ------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return tuple(_exact_rotary(case, s[x], s["positions"]) for x in ("q", "k"))
    if case["op"] == "prompt":
        return _exact_prompt(case, s)
    if case["op"] == "store":
        return tuple(_exact_held(s[x]) for x in ("k", "v"))
    d, n = case["d"], case["n"]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        for i in range(n):
            sees = L - (n - 1 - i)
            if sees <= 0:
                continue
            for j in range(case["heads"]):
                g = j // group
                kk, vv = (s["codes_" + x][b, g, :sees].double().view(sees, -1, 32) *
                          s["scales_" + x][b, g, :sees].double()[..., None] for x in ("k", "v"))
                p = torch.softmax(kk.view(sees, d) @ s["q"][b, j, i].double() / math.sqrt(d), 0)
                out[b, j, i] = p @ vv.view(sees, d)
    return out


def _exact_rotary(case, x, positions):
    """Pair by pair, as a product with a unit complex number."""
    out = x.double().clone()
    P = sum(_sections(case))
    p = 0
    for axis, count in enumerate(_sections(case)):
        for i in range(count):
            a, b = (p, P + p) if case["pairing"] == "halves" else (2 * p, 2 * p + 1)
            angle = positions[axis].double() * math.pow(_BASE, -i / count)
            angle = -angle if case["dir"] == "bwd" else angle
            if angle.dim() == 2:
                angle = angle[:, None]
            z = torch.complex(x[..., a].double(), x[..., b].double()) * torch.polar(torch.ones_like(angle), angle)
            out[..., a], out[..., b] = z.real, z.imag
            p += 1
    return out


def _exact_held(x):
    """Values that the cache stands for.  A 64-bit quotient of two fp32 numbers rounded to fp32 is the fp32 quotient."""
    x = x.double()
    out = torch.empty_like(x)
    for c in range(0, x.shape[-1], 32):
        part = x[..., c:c + 32]
        scale = (part.abs().max(-1, keepdim=True).values / 7).float().to(torch.bfloat16).double()
        code = torch.round((part / scale).float()).double()
        out[..., c:c + 32] = torch.where(scale > 0, code * scale, 0.0)
    return out


def _exact_prompt(case, s):
    h, d, train = case["heads"], case["d"], case["dir"] == "train"
    group = h // case["kv_heads"]
    out = torch.zeros(h, s["q"].shape[1], d, dtype=torch.float64, device="cuda")
    if train:
        dq, dk, dv = torch.zeros_like(out), *(torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
                                              for _ in range(2))
    start = 0
    for L in _prompt_lengths(case):
        step = max(1, (1 << 26) // max(L, 1))
        for j in range(h):
            g = j // group
            for i in range(0, L, step):
                n = min(step, L - i)
                last = i + n if case["causal"] else L          # keys that these rows can see
                rows, keys = slice(start + i, start + i + n), slice(start, start + last)
                q, k, v = s["q"][j, rows].double(), s["k"][g, keys].double(), s["v"][g, keys].double()
                x = q @ k.T / math.sqrt(d)
                if case["causal"]:
                    at = torch.arange(last, device="cuda")
                    x = torch.where(at[None, :] <= at[i:last, None], x, -math.inf)
                p = torch.softmax(x, -1)
                out[j, rows] = p @ v
                if train:
                    up = s["dout"][j, rows].double()
                    dv[g, keys] += p.T @ up
                    dx = up @ v.T
                    dx = p * (dx - (p * dx).sum(-1, keepdim=True))
                    dq[j, rows] = dx @ k / math.sqrt(d)
                    dk[g, keys] += dx.T @ q / math.sqrt(d)
        start += L
    return (out, dq, dk, dv) if train else out
