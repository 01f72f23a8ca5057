"""The cross attention and the relative position bias on the GPU against their
64-bit restatement, elementwise within the bounds derived there
(attention_ref.py); determinism, streams, graphs, masked garbage."""
import math

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def lisa():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from hop_stochastic_vision_gb300 import build, lisa as binding
    build.build()
    binding.load()
    return binding


def _rule(lisa, r):
    return lisa.exact_buckets(r[1]) if r[0] == "exact" else lisa.log_buckets(r[1], r[2])


class Case:
    def __init__(self, lisa, dtype, B, heads, kv, n, m, d, *, bias=None, lens=None, layout="heads", scale=None, seed=0,
                 spread=1.0, garbage=False):
        g = torch.Generator().manual_seed(seed)
        q_grid, k_grid = (n if isinstance(n, tuple) else (1, n)), (m if isinstance(m, tuple) else (1, m))
        n, m = q_grid[0] * q_grid[1], k_grid[0] * k_grid[1]
        self.lisa, self.dtype, self.scale = lisa, dtype, 1 / math.sqrt(d) if scale is None else scale
        q = (spread * torch.randn(B, heads, n, d, generator=g)).to(dtype)
        k, v = (torch.randn(B, kv, m, d, generator=g).to(dtype) for _ in range(2))
        self.dout = torch.randn(B, heads, n, d, generator=g).to(dtype)
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32)
        self.k_ref, self.v_ref = k.clone(), v.clone()
        if garbage:
            for b, L in enumerate(lens):
                k[b, :, max(L, 0):], v[b, :, max(L, 0):] = math.nan, math.inf
        self.q_ref = q
        if layout == "tokens":      # [B, tokens, heads, d], keys beside values
            self.q = q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
            pair = torch.stack((k.transpose(1, 2), v.transpose(1, 2)), 2).contiguous().cuda()
            self.k, self.v = pair[:, :, 0].transpose(1, 2), pair[:, :, 1].transpose(1, 2)
            self.do = self.dout.cuda().transpose(1, 2).contiguous().transpose(1, 2)
        else:
            self.q, self.k, self.v, self.do = q.cuda(), k.cuda(), v.cuda(), self.dout.cuda()
        self.bias = self.index = self.table = None
        if bias is not None:
            rows, cols = bias.get("rows", ("exact", 0)), bias["cols"]
            step, start = bias.get("step", (1, 1)), bias.get("start", (0, 0))
            self.table = torch.randn(ref.buckets(rows) * ref.buckets(cols), heads, generator=g)
            for row in bias.get("minus_inf", ()):
                self.table[row] = -math.inf
            self.index = ref.bucket_index(q_grid, k_grid, rows, cols, step, start)
            self.bias = lisa.RelativeBias(self.table.cuda(), q_grid, k_grid, rows=_rule(lisa, rows),
                                          cols=_rule(lisa, cols), key_step=step, query_start=start)
        self.kw = dict(scale=self.scale, kv_lens=None if self.lens is None else self.lens.cuda(), bias=self.bias)

    def want(self, backward=True):
        return ref.attention(self.q_ref, self.k_ref, self.v_ref, self.dout if backward else None, scale=self.scale,
                             lens=None if self.lens is None else self.lens.tolist(), table=self.table,
                             index=self.index, dtype=self.dtype)

    def forward(self, **kw):
        return self.lisa.cross_attention(self.q, self.k, self.v, return_lse=True, **{**self.kw, **kw})

    def backward(self, out, lse, **kw):
        return self.lisa.cross_attention_backward(self.q, self.k, self.v, out, lse, self.do, **{**self.kw, **kw})

    def check(self):
        out, lse = self.forward()
        grads = self.backward(out, lse)
        want = self.want()
        for name, got in zip(("o", "lse", "dq", "dk", "dv", "dtable"), (out, lse) + tuple(grads)):
            ref.assert_within(got, want[name], name)
        assert len(grads) == (3 if self.bias is None else 4)
        return out, lse, grads


LOG = {"cols": ("log", 32, 128)}
SHORT = {"cols": ("log", 8, 5), "start": (0, 3)}
NEAR = {"cols": ("exact", 3), "start": (0, -2)}


def _grid(q, k, step=1, **kw):
    D = [max(a - 1, step * (b - 1)) for a, b in zip(q, k)]
    return {"rows": ("exact", D[0]), "cols": ("exact", D[1]), "step": (step, step), **kw}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("n,m", [(1, 1), (1, 7), (5, 1), (17, 200), (64, 64), (65, 63), (129, 130), (257, 49)])
def test_lengths_and_widths(lisa, dtype, d, n, m):
    Case(lisa, dtype, 2, 2, 1, n, m, d, seed=n + m).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads,kv", [(4, 4), (4, 2), (6, 1), (3, 3)])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_head_layouts(lisa, dtype, heads, kv, layout):
    Case(lisa, dtype, 3, heads, kv, 70, 150, 64, layout=layout, seed=heads).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bias", [None, LOG, SHORT])
@pytest.mark.parametrize("garbage", [False, True])
def test_padded_batches(lisa, dtype, bias, garbage):
    """Lengths of 0 and 1, ends inside and at a tile; what stands behind them (NaN, inf) plays no part."""
    Case(lisa, dtype, 6, 2, 1, 90, 300, 64, bias=bias, lens=[0, 1, 128, 129, 299, 300], garbage=garbage).check()


def test_lengths_outside_the_range_count_as_its_ends(lisa):
    c = Case(lisa, BF16, 3, 2, 2, 20, 40, 64, lens=[-5, 40, 1000])
    c.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bias", [LOG, SHORT, NEAR, {"cols": ("exact", 300)}, {"cols": ("log", 128, 1000)},
                                  {"cols": ("log", 4, 2), "step": (1, 3)}, {"cols": ("exact", 40), "start": (0, 90)}])
def test_sequence_biases(lisa, dtype, bias):
    Case(lisa, dtype, 2, 4, 2, 140, 200, 64, bias=bias, seed=3).check()


@pytest.mark.parametrize("dtype,d", [(F32, 16), (F32, 64), (BF16, 64), (BF16, 32)])
@pytest.mark.parametrize("q,k,step", [((14, 14), (14, 14), 1), ((7, 9), (3, 5), 2), ((12, 20), (2, 3), 8),
                                      ((1, 5), (4, 1), 1), ((5, 1), (1, 6), 3), ((17, 23), (17, 23), 1)])
def test_grid_biases(lisa, dtype, d, q, k, step):
    Case(lisa, dtype, 3, 2, 2, q, k, d, bias=_grid(q, k, step), seed=step).check()


def test_the_largest_offset_table(lisa):
    """16296 offsets and as many keys: the shared memory of every kernel at its fullest."""
    c = Case(lisa, BF16, 1, 1, 1, (1, 1), (168, 97), 64, bias=_grid((1, 1), (168, 97)))
    c.check()
    Case(lisa, BF16, 1, 1, 1, (64, 64), (8, 8), 64, bias=_grid((64, 64), (8, 8), 8)).check()


def test_an_offset_table_that_fills_the_shared_memory(lisa):
    """32 KB of offsets: with whole stages of tiles the dQ kernel's memory to the last KB."""
    Case(lisa, BF16, 1, 1, 1, 3900, 3900, 64, bias={"cols": ("exact", 3850)}).check()


@pytest.mark.parametrize("m", [1, 2, 3, 128])
def test_few_keys_keep_small_differences(lisa, m):
    """One tile of keys: delta is the sum of the unrounded p dP, so dQ = scale sum dS k is
    good to the rounding of dS and of dQ alone, however much of dP - delta cancels."""
    for bias in (None, {"cols": ("exact", 2)}):
        c = Case(lisa, BF16, 3, 2, 2, 40, m, 64, bias=bias, spread=4.0)
        out, lse = c.forward()
        dq = c.backward(out, lse)[0].double().cpu()
        s = c.q_ref.double() @ c.k_ref.double().transpose(-1, -2) * c.scale
        if bias:
            s = s + c.table.double().t()[:, c.index]
        p = torch.softmax(s, -1)
        dp = c.dout.double() @ c.v_ref.double().transpose(-1, -2)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        want = c.scale * ds @ c.k_ref.double()
        mag = c.scale * ds.abs() @ c.k_ref.double().abs()
        # dS and dQ rounded, half a step 2^-8 each; behind them fp32: s of magnitude up to 150 with a few 2^-24 of it in
        # the exponent (2^-14 of p), dP - delta with 64 2^-24 of |dO| |v| (below 2^-12 of sum |dO v|), both of p dP
        noise = c.scale * ((p * (2.0 ** -14 * (dp.abs() + (p * dp).abs().sum(-1, keepdim=True)) + 2.0 ** -16 * (
            c.dout.double().abs() @ c.v_ref.double().abs().transpose(-1, -2)))) @ c.k_ref.double().abs())
        assert ((dq - want).abs() <= (2.0 ** -8 + 2.0 ** -8 * 1.01) * mag + noise + 2.0 ** -126).all()


def test_grid_bias_with_near_and_far_offsets_in_one_bucket(lisa):
    q, k = (9, 11), (6, 7)
    for rows, cols in ((("exact", 2), ("log", 8, 5)), (("log", 16, 9), ("exact", 0))):
        Case(lisa, BF16, 2, 3, 1, q, k, 64, bias={"rows": rows, "cols": cols, "step": (2, 1), "start": (1, -2)}).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_buckets_of_minus_infinity_mask(lisa, dtype):
    """-inf table entries mask pairs, here whole rows too: o = 0, lse = -inf, no gradient, no NaN."""
    bias = {"cols": ("exact", 2), "minus_inf": (0, 4)}      # offsets of 2 and more are masked
    c = Case(lisa, dtype, 2, 2, 2, 150, 140, 64, bias=bias)
    out, lse, grads = c.check()
    assert torch.isinf(lse[:, :, 142:]).all() and not out[:, :, 142:].any() and not grads[0][:, :, 142:].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores(lisa, dtype):
    """Scores of some hundreds: the maximum moves between tiles and the sum is rescaled."""
    Case(lisa, dtype, 1, 2, 2, 100, 500, 64, spread=12.0, scale=1.0).check()


def test_repeated_inputs(lisa):
    """One set of states for the whole batch (stride 0), and one key head for all: dk, dv of the repeated tensor."""
    c = Case(lisa, BF16, 3, 2, 2, 60, 80, 64)
    c.k, c.v = c.k[:1].expand(3, -1, -1, -1), c.v[:1].expand(3, -1, -1, -1)
    c.k_ref, c.v_ref = c.k.cpu(), c.v.cpu()
    c.check()
    c = Case(lisa, F32, 2, 4, 4, 33, 41, 32)
    c.k, c.v = c.k[:, :1].expand(-1, 4, -1, -1), c.v[:, :1].expand(-1, 4, -1, -1)
    c.k_ref, c.v_ref = c.k.cpu(), c.v.cpu()
    c.check()


def test_no_keys_at_all(lisa):
    q = torch.randn(2, 3, 5, 64, device="cuda", dtype=BF16)
    k = torch.empty(2, 3, 0, 64, device="cuda", dtype=BF16)
    out, lse = lisa.cross_attention(q, k, k, return_lse=True)
    assert not out.any() and torch.isinf(lse).all() and (lse < 0).all()
    dq, dk, dv = lisa.cross_attention_backward(q, k, k, out, lse, q)
    assert not dq.any() and dk.shape == k.shape and dv.shape == k.shape


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_keys_into_a_given_layout(lisa, dtype):
    q = torch.randn(2, 3, 700, 32, device="cuda", dtype=dtype)
    k = torch.empty(2, 1, 0, 32, device="cuda", dtype=dtype)
    wide = torch.full((2, 700, 4, 32), 7.0, dtype=dtype, device="cuda")
    lisa.cross_attention(q, k, k, out=wide[:, :, :3].transpose(1, 2))
    assert not wide[:, :, :3].any() and (wide[:, :, 3] == 7).all()
    _, lse = lisa.cross_attention(q, k, k, return_lse=True)
    assert (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,heads,kv,m", [(1, 1, 1, 1), (1, 3, 3, 196), (5, 8, 2, 1000), (3, 16, 1, 130),
                                          (40, 4, 4, 63), (1, 12, 4, 4097), (2, 24, 1, 600)])
def test_single_tokens(lisa, dtype, B, heads, kv, m):
    lens = None if B == 1 else [(m * b) // (B - 1) for b in range(B)]
    for d in (16, 64):
        c = Case(lisa, dtype, B, heads, kv, 1, m, d, lens=lens, layout="tokens" if d == 64 else "heads",
                 garbage=lens is not None)
        want = c.want(backward=False)
        out, lse = c.forward()
        ref.assert_within(out, want["o"], "o")
        ref.assert_within(lse, want["lse"], "lse")


@pytest.mark.parametrize("n", [2, 3, 8, 16, 40])
def test_few_tokens_over_many_keys(lisa, n):
    c = Case(lisa, BF16, 2, 4, 2, n, 2500, 64, lens=[2500, 777], bias={"cols": ("log", 32, 128), "start": (0, 2000)})
    want = c.want(backward=False)
    out, lse = c.forward()
    ref.assert_within(out, want["o"], "o")
    ref.assert_within(lse, want["lse"], "lse")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens_at_their_own_positions(lisa, dtype):
    B, heads, m = 4, 6, 900
    c = Case(lisa, dtype, B, heads, 2, 1, m, 64, lens=[900, 3, 500, 0])
    starts = [0, 899, -7, 5]
    rule = ("log", 32, 128)
    table = torch.randn(32, heads)
    c.table, c.index = table, [ref.bucket_index((1, 1), (1, m), ("exact", 0), rule, (1, 1), (0, s)) for s in starts]
    c.bias = lisa.RelativeBias(table.cuda(), (1, 1), (1, m), cols=_rule(lisa, rule),
                               query_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    out, lse = c.forward(bias=c.bias)
    want = c.want(backward=False)
    ref.assert_within(out, want["o"], "o")
    ref.assert_within(lse, want["lse"], "lse")
    with pytest.raises(ValueError):
        c.backward(out, lse, bias=c.bias)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_every_time_whatever_the_workspace_holds(lisa, dtype):
    from hop_stochastic_vision_gb300 import attention as att
    c = Case(lisa, dtype, 3, 4, 2, (10, 13), (10, 13), 64, bias=_grid((10, 13), (10, 13)), lens=[130, 55, 0])
    dt = lisa.LISA_F32 if dtype == F32 else lisa.LISA_BF16
    out, lse = c.forward()
    first = c.backward(out, lse)
    for fill in (0x00, 0xFF):
        nf = att.lisa_cross_attention_workspace_bytes(3, 4, 2, 130, 130, 64, c.bias.struct, dt)
        nb = att.lisa_cross_attention_backward_workspace_bytes(3, 4, 2, 130, 130, 64, c.bias.struct, dt)
        ws = torch.full((max(nf, nb, 16),), fill, dtype=torch.uint8, device="cuda")
        out2, lse2 = c.forward(workspace=ws)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        ws.fill_(fill)
        for a, b in zip(first, c.backward(out, lse, workspace=ws)):
            assert torch.equal(a, b)


def test_a_given_output_is_written_in_its_own_layout_and_nothing_else(lisa):
    c = Case(lisa, BF16, 2, 3, 3, 37, 90, 64)
    wide = torch.full((2, 40, 4, 64), 7.0, dtype=BF16, device="cuda")       # rows and a head to spare
    view = wide[:, :37, :3].transpose(1, 2)
    res = lisa.cross_attention(c.q, c.k, c.v, out=view, **c.kw)
    assert res is view
    assert torch.equal(view, c.forward()[0])
    assert (wide[:, 37:] == 7).all() and (wide[:, :, 3] == 7).all()


def test_other_streams_and_captured_graphs(lisa):
    c = Case(lisa, BF16, 2, 4, 2, 100, 260, 64, bias=LOG, lens=[260, 100])
    out, lse = c.forward()
    grads = c.backward(out, lse)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, l2 = c.forward()
        g2 = c.backward(o2, l2)
    o3, l3 = c.forward(stream=side.cuda_stream)
    g3 = c.backward(o3, l3, stream=side.cuda_stream)
    side.synchronize()
    for a, b, x in zip((out, lse) + grads, (o2, l2) + g2, (o3, l3) + g3):
        assert torch.equal(a, b) and torch.equal(a, x)
    # captured, replayed on two inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = c.forward()
        gg = c.backward(og, lg)
    for seed in (0, 9):
        other = Case(lisa, BF16, 2, 4, 2, 100, 260, 64, bias=LOG, lens=[260, 100], seed=seed)
        for name in ("q", "k", "v", "do"):
            getattr(c, name).copy_(getattr(other, name))
        c.bias.table.copy_(other.bias.table)
        graph.replay()
        torch.cuda.synchronize()
        oe, le = other.forward()
        for a, b in zip((og, lg) + gg, (oe, le) + other.backward(oe, le)):
            assert torch.equal(a, b)


def test_gradient_against_differences(lisa):
    """fp32 directional derivatives by central differences.  With L = sum(o dO)
    and a unit step of h along x the difference quotient is off by h^2 / 6 times
    the third derivative (of the order of L's scale: 3e-6 at h = 2^-8) and by
    the rounding of the two sums, at most 2^-23 sum|o dO| (m + d) / h."""
    c = Case(lisa, F32, 2, 2, 1, 24, 30, 16, bias={"cols": ("exact", 4)})
    out, lse = c.forward()
    grads = c.backward(out, lse)
    h = 2.0 ** -8
    for x, dx in zip((c.q, c.k, c.v, c.bias.table), grads):
        dirn = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda()
        dirn /= dirn.norm()
        keep, vals = x.clone(), []
        for sign in (1, -1):
            x.copy_(keep + sign * h * dirn)
            vals.append((c.forward()[0].double() * c.do.double()).sum())
        x.copy_(keep)
        got, want = float((dx.double() * dirn.double()).sum()), float((vals[0] - vals[1]) / (2 * h))
        scale = float((out.abs().double() * c.do.abs().double()).sum())
        assert abs(got - want) <= h * h * scale + 2.0 ** -23 * scale * (30 + 16) / h


LOWEST = (torch.finfo(F32).min, torch.finfo(BF16).min)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 150])
def test_the_types_lowest_values_mask(lisa, dtype, n):
    """Entries of the lowest finite value mask as -inf does, on every path, rows that they leave empty too."""
    c = Case(lisa, dtype, 2, 2, 2, n, 140, 64, bias={"cols": ("exact", 2), "start": (0, 0 if n > 1 else 137),
                                                     "minus_inf": (0, 4)})
    want = c.want(backward=n > 1)
    for e, row in enumerate((0, 4)):
        c.bias.table[row] = LOWEST[e]
    out, lse = c.forward()
    ref.assert_within(out, want["o"], "o")
    ref.assert_within(lse, want["lse"], "lse")
    if n > 1:
        assert torch.isinf(lse[:, :, 142:]).all() and not out[:, :, 142:].any()
        for name, got in zip(("dq", "dk", "dv", "dtable"), c.backward(out, lse)):
            ref.assert_within(got, want[name], name)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_masked_by_large_finite_numbers(lisa, dtype):
    """-1e9 over a whole row leaves fp32 nothing of the scores: finite outputs, and
    the gradients are those of a row without keys (rows 141 and on: offsets of -2 and less)."""
    c = Case(lisa, dtype, 2, 2, 2, 150, 140, 64, bias={"cols": ("exact", 2), "minus_inf": (0, 4)})
    out, lse = c.forward()
    want = c.backward(out, lse)
    for row in (0, 4):
        c.bias.table[row] = -1e9
    o2, l2 = c.forward()
    assert torch.isfinite(o2).all() and torch.equal(o2[:, :, :141], out[:, :, :141])
    assert torch.isfinite(l2).all() and torch.equal(l2[:, :, :141], lse[:, :, :141])
    for a, b in zip(c.backward(o2, l2), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_error_word_is_cleared(lisa, dtype):
    from hop_stochastic_vision_gb300 import attention as att
    c = Case(lisa, dtype, 2, 2, 2, 70, 90, 64)
    dt = lisa.LISA_F32 if dtype == F32 else lisa.LISA_BF16
    stream = torch.cuda.current_stream().cuda_stream
    out, lse = c.forward()
    sizes = (att.lisa_cross_attention_workspace_bytes(2, 2, 2, 70, 90, 64, None, dt),
             att.lisa_cross_attention_backward_workspace_bytes(2, 2, 2, 70, 90, 64, None, dt))
    for nbytes, call in zip(sizes, (lambda w: c.forward(workspace=w), lambda w: c.backward(out, lse, workspace=w))):
        if nbytes:
            ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
            call(ws)
            assert lisa.lisa_query_status(ws.data_ptr(), stream) == lisa.LISA_OK


@pytest.mark.parametrize("dtype,n", [(F32, 70), (BF16, 70), (BF16, 1)])
def test_offsets_beyond_32_bits(lisa, dtype, n):
    """Keys a million elements apart: the last ones stand 2^31 elements and more from the first."""
    m, gap = 2200, 1 << 20
    c = Case(lisa, dtype, 1, 1, 1, n, m, 64)
    out, lse = c.forward()
    grads = c.backward(out, lse)
    wide = torch.empty(m * gap, dtype=dtype, device="cuda").view(1, 1, m, gap)
    for at, name in ((0, "k"), (64, "v")):
        wide[..., at:at + 64] = getattr(c, name)
        setattr(c, name, wide[..., at:at + 64])
    o2, l2 = c.forward()
    for a, b in zip((out, lse) + grads, (o2, l2) + c.backward(o2, l2)):
        assert torch.equal(a, b)


def test_the_most_queries(lisa):
    """2^22 queries of two keys, fp32 with a bias: more tiles than a grid's second axis holds."""
    n = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(0)
    q, do = (torch.randn(1, 1, n, 16, generator=g, device="cuda") for _ in range(2))
    k, v = (torch.randn(1, 1, 2, 16, generator=g, device="cuda") for _ in range(2))
    table = torch.randn(3, 1, generator=g, device="cuda")
    bias = lisa.RelativeBias(table, (1, n), (1, 2), cols=lisa.exact_buckets(1))
    out, lse = lisa.cross_attention(q, k, v, bias=bias, return_lse=True)
    dtable = lisa.cross_attention_backward(q, k, v, out, lse, do, bias=bias)[3]
    s = q[0, 0].double() @ k[0, 0].double().t() / 4 + table.double()[0, 0]
    s[:2] = q[0, 0, :2].double() @ k[0, 0].double().t() / 4 + table.double()[[[1, 2], [0, 1]], 0]
    p = torch.softmax(s, -1)
    dp = do[0, 0].double() @ v[0, 0].double().t()
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    want = torch.stack((ds[2:].sum() + ds[1, 0], ds[0, 0] + ds[1, 1], ds[0, 1]))
    # a term is off by a few 2^-24 of the scores' and dP's magnitudes (|s| to 30, |dP| to 60: 64 of them), the sum of
    # the n terms in runs of at most 2^13 by 2^-24 2^13 of the terms' magnitude
    bound = 2.0 ** -24 * (64 * 30 + 2 ** 13) * ds.abs().sum()
    assert ((dtable[:, 0].double() - want).abs() <= bound).all()
    assert (out[0, 0].double() - p @ v[0, 0].double()).abs().max() <= 2.0 ** -24 * 64 * 30 * v.abs().max()


def test_two_graphs_share_a_workspace(lisa):
    from hop_stochastic_vision_gb300 import attention as att
    cases = [Case(lisa, BF16, 2, 4, 2, n, 260, 64, bias=LOG, seed=n) for n in (100, 333)]
    nbytes = max(att.lisa_cross_attention_backward_workspace_bytes(2, 4, 2, n, 260, 64, c.bias.struct, lisa.LISA_BF16)
                 for n, c in zip((100, 333), cases))
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    want, graphs, got = [], [], []
    for c in cases:
        out, lse = c.forward()
        want.append((out, lse) + c.backward(out, lse))
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            out, lse = c.forward(workspace=ws)
            got.append((out, lse) + c.backward(out, lse, workspace=ws))
    for which in (0, 1, 1, 0, 1):
        for x in got[which]:
            x.fill_(7)
        graphs[which].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[which], want[which]))


def test_calls_side_by_side(lisa):
    """Calls on two streams at once, each with its own workspace."""
    cases = [Case(lisa, BF16, 4, 4, 2, 500, 600, 64, bias=LOG, seed=s) for s in (1, 2)]
    want = []
    for c in cases:
        out, lse = c.forward()
        want.append((out, lse) + c.backward(out, lse))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], [[], []]
    for _ in range(8):
        for c, s, res in zip(cases, streams, got):
            with torch.cuda.stream(s):
                out, lse = c.forward()
                res.append((out, lse) + c.backward(out, lse))
    torch.cuda.synchronize()
    for res, w in zip(got, want):
        assert all(torch.equal(a, b) for r in res for a, b in zip(r, w))


def test_a_table_that_moved(lisa):
    c = Case(lisa, BF16, 1, 2, 2, 40, 50, 64, bias=NEAR)
    out = c.forward()[0]
    c.bias.table.data = c.bias.table.clone()
    assert torch.equal(c.forward()[0], out)
    c.bias.table = c.bias.table.cpu()
    with pytest.raises(ValueError):
        c.forward()


def test_refusals(lisa):
    q, k = (torch.randn(2, 2, n, 64, device="cuda", dtype=BF16) for n in (8, 9))
    ok = lisa.cross_attention(q, k, k)
    bad = [(q.float(), k, k), (q, k[:, :, :8], k), (q, k, k.float()), (q, k.cpu(), k), (q[0], k, k), (q.half(), k, k),
           (q, k.transpose(2, 3).contiguous().transpose(2, 3), k), (q[:1], k, k)]
    for args in bad:
        with pytest.raises(ValueError):
            lisa.cross_attention(*args)
    off = torch.randn(2 * 2 * 8 * 64 + 1, device="cuda", dtype=BF16)[1:].view(2, 2, 8, 64)     # 2 bytes off
    narrow = torch.randn(2, 2, 8, 40, device="cuda", dtype=BF16)
    none = torch.empty(2, 2, 8, 0, device="cuda", dtype=BF16)
    odd = torch.randn(2, 2, 8, 68, device="cuda", dtype=BF16)[..., :64]                       # rows of 136 bytes
    for args in ((off, k, k), (narrow, narrow, narrow), (none, none, none), (odd, k, k), (q, q[:, :, :0], q[:, :, :1])):
        with pytest.raises((lisa.LisaError, ValueError)):
            lisa.cross_attention(*args)
    with pytest.raises(lisa.LisaError):
        lisa.cross_attention(q, k, k, out=q)
    with pytest.raises(lisa.LisaError):
        lisa.cross_attention(q, k, k, scale=-1.0)
    with pytest.raises(lisa.LisaError):
        lisa.cross_attention(q, q.new_empty(2, 3, 9, 64), q.new_empty(2, 3, 9, 64))            # 2 heads over 3
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    out, lse = lisa.cross_attention(torch.cat((q,) * 8, 2), k, k, return_lse=True)
    with pytest.raises(lisa.LisaError):
        lisa.cross_attention(torch.cat((q,) * 8, 2), k, k, workspace=small)
    with pytest.raises(ValueError):
        lisa.cross_attention_backward(q, k, k, ok, lse, q)                                     # another call's lse
    for lens in (torch.ones(2, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda"),
                 torch.ones(2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            lisa.cross_attention(q, k, k, kv_lens=lens)
    table = torch.zeros(32, 2, device="cuda")
    with pytest.raises(ValueError):
        lisa.cross_attention(q, k, k, bias=lisa.RelativeBias(table, (1, 8), (1, 8), cols=lisa.log_buckets(32, 128)))
    for args in ((table[:31], (1, 8), (1, 9)), (table.double(), (1, 8), (1, 9)), (table.t(), (1, 8), (1, 9)),
                 (table.cpu(), (1, 8), (1, 9))):
        with pytest.raises(ValueError):
            lisa.RelativeBias(*args, cols=lisa.log_buckets(32, 128))
    assert torch.equal(lisa.cross_attention(q, k, k), ok)


# ------------------------------------------------------------------ the bias matrix

MATRICES = [((1, 1), (1, 1), LOG), ((1, 50), (1, 77), LOG), ((1, 300), (1, 5), SHORT), ((1, 40), (1, 600), NEAR),
            ((1, 33), (1, 20), {"cols": ("log", 16, 60), "step": (1, 5)}), ((14, 14), (14, 14), None),
            ((24, 24), (24, 24), None), ((13, 7), (3, 2), 4), ((7, 30), (7, 30), None),
            ((6, 5), (9, 4), {"rows": ("log", 8, 4), "cols": ("exact", 1), "step": (2, 3), "start": (-1, 2)}),
            ((1, 900), (1, 1100), {"cols": ("exact", 700)}),
            ((1, 1000), (1, 1500), {"cols": ("exact", 8), "step": (1, 300), "start": (0, 40000)}),
            ((1, 90), (1, 40), {"cols": ("log", 8, 5), "step": (1, 5000), "start": (0, 60)})]


def _matrix(lisa, q, k, how, heads=3):
    bias = _grid(q, k, how if isinstance(how, int) else 1) if how is None or isinstance(how, int) else how
    rows, cols = bias.get("rows", ("exact", 0)), bias["cols"]
    step, start = bias.get("step", (1, 1)), bias.get("start", (0, 0))
    table = torch.randn(ref.buckets(rows) * ref.buckets(cols), heads, generator=torch.Generator().manual_seed(2))
    b = lisa.RelativeBias(table.cuda(), q, k, rows=_rule(lisa, rows), cols=_rule(lisa, cols), key_step=step,
                          query_start=start)
    return b, table, ref.bucket_index(q, k, rows, cols, step, start)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("q,k,how", MATRICES)
def test_bias_matrix(lisa, dtype, q, k, how):
    b, table, index = _matrix(lisa, q, k, how)
    got = lisa.relative_bias(b, dtype)
    assert torch.equal(got.cpu(), table.t()[:, index].to(dtype))      # table values, rounded once
    wide = torch.full((got.numel() + 64,), 3.0, dtype=dtype, device="cuda")
    out = wide[16:16 + got.numel()].view(got.shape)
    assert torch.equal(lisa.relative_bias(b, dtype, out=out), got)
    assert (wide[:16] == 3).all() and (wide[16 + got.numel():] == 3).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("q,k,how", MATRICES)
def test_bias_matrix_gradient(lisa, dtype, q, k, how):
    """fp32 sums of N terms in any order are within N 2^-24 sum|x|; a bucket without pairs gives 0."""
    b, table, index = _matrix(lisa, q, k, how)
    heads, n, m = 3, b.n, b.m
    x = torch.randn(heads, n, m, generator=torch.Generator().manual_seed(4)).to(dtype)
    got = lisa.relative_bias_backward(b, x.cuda()).cpu().double()
    want, mag, count = (torch.zeros(table.shape, dtype=torch.float64) for _ in range(3))
    for h in range(heads):
        want[:, h].index_add_(0, index.reshape(-1), x[h].reshape(-1).double())
        mag[:, h].index_add_(0, index.reshape(-1), x[h].reshape(-1).double().abs())
        count[:, h].index_add_(0, index.reshape(-1), torch.ones(n * m, dtype=torch.float64))
    assert ((got - want).abs() <= count * 2.0 ** -24 * mag).all()
    again = lisa.relative_bias_backward(b, x.cuda(), workspace=torch.full((1 << 24,), 0xFF, dtype=torch.uint8,
                                                                          device="cuda"))
    assert torch.equal(again.cpu().double(), got)


def test_bias_of_infinities(lisa):
    b, table, index = _matrix(lisa, (1, 20), (1, 20), LOG)
    b.table[3] = -math.inf
    table[3] = -math.inf
    assert torch.equal(lisa.relative_bias(b).cpu(), table.t()[:, index])


# ------------------------------------------------------------------ as a layer uses them

def test_a_pooled_stage_beside_the_linear_layer(lisa):
    """One stage as a backbone runs it: the LiSA layer on a 16 x 16 grid, its
    output as the queries of a pooled attention with a learned bias, trained by
    both backward passes; the fused bias agrees with the matrix added by hand."""
    g = torch.Generator().manual_seed(11)
    B, heads, H, W, d = 2, 2, 16, 16, 64
    xq, xk, v, do = (torch.randn(B, heads, H * W, d, generator=g).to(BF16).cuda() for _ in range(4))
    alpha = torch.full((heads,), 0.5).cuda()
    layer = lisa.forward(xq, xk, v, (H, W), 3, alpha=alpha, beta=0.5)
    pooled = layer.float().reshape(B, heads, 4, 4, 4, 4, d).mean((3, 5)).reshape(B, heads, 16, d).to(BF16)
    rule = _grid((H, W), (4, 4), 4)
    table = torch.randn(ref.buckets(rule["rows"]) * ref.buckets(rule["cols"]), heads, generator=g).cuda()
    bias = lisa.RelativeBias(table, (H, W), (4, 4), rows=_rule(lisa, rule["rows"]), cols=_rule(lisa, rule["cols"]),
                             key_step=(4, 4))
    out, lse = lisa.cross_attention(layer, pooled, pooled, bias=bias, return_lse=True)
    dq, dk, dv, dtable = lisa.cross_attention_backward(layer, pooled, pooled, out, lse, do, bias=bias)
    index = ref.bucket_index((H, W), (4, 4), rule["rows"], rule["cols"], (4, 4))
    want = ref.attention(layer, pooled, pooled, do, scale=1 / 8, table=table, index=index)
    for name, got in (("o", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv), ("dtable", dtable)):
        ref.assert_within(got, want[name], name)
    # dS of the whole batch through the matrix's own gradient
    matrix = lisa.relative_bias(bias).double()
    p = torch.softmax(layer.double() @ pooled.double().transpose(-1, -2) / 8 + matrix, -1)
    dp = do.double() @ pooled.double().transpose(-1, -2)
    ds = (p * (dp - (p * dp).sum(-1, keepdim=True))).sum(0).float()
    by_matrix = lisa.relative_bias_backward(bias, ds)
    ref.assert_within(by_matrix, (want["dtable"][0], want["dtable"][1] + 2.0 ** -24 * 256 * 16 * ds.abs().max().cpu()),
                      "dtable by the matrix")
    grads = lisa.backward(xq, xk, v, dq, (H, W), 3, alpha=alpha, beta=0.5)
    assert all(torch.isfinite(x).all() for x in grads)


def test_bias_matrix_refusals(lisa):
    b, _, _ = _matrix(lisa, (1, 20), (1, 24), LOG)
    own = lisa.RelativeBias(b.table, (1, 1), (1, 24), cols=lisa.log_buckets(32, 128),
                            query_start=torch.zeros(4, dtype=torch.int32, device="cuda"))
    good = torch.zeros(3, 20, 24, device="cuda")
    for call in (lambda: lisa.relative_bias(b, torch.float16), lambda: lisa.relative_bias(own),
                 lambda: lisa.relative_bias(b, out=good.to(BF16)), lambda: lisa.relative_bias(b, out=good[:, :, :23]),
                 lambda: lisa.relative_bias(b, out=good.cpu()), lambda: lisa.relative_bias_backward(b, good.double()),
                 lambda: lisa.relative_bias_backward(b, good[:2]), lambda: lisa.relative_bias_backward(b, good.cpu()),
                 lambda: lisa.relative_bias_backward(b, good.transpose(1, 2).contiguous().transpose(1, 2)),
                 lambda: lisa.relative_bias_backward(own, good)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(lisa.LisaError):       # too small a workspace
        lisa.relative_bias_backward(b, good, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    far = lisa.RelativeBias(torch.zeros(129 * 129, 3, device="cuda"), (65, 65), (65, 65), rows=lisa.exact_buckets(64),
                            cols=lisa.exact_buckets(64))
    with pytest.raises(lisa.LisaError):       # more offsets than the shared memory holds
        lisa.relative_bias(far)


def test_empty_batches(lisa):
    for dtype in (F32, BF16):
        q, k = torch.empty(0, 2, 5, 64, device="cuda", dtype=dtype), torch.empty(0, 1, 9, 64, device="cuda", dtype=dtype)
        table = torch.randn(7, 2, device="cuda")
        bias = lisa.RelativeBias(table, (1, 5), (1, 9), cols=lisa.exact_buckets(3))
        out, lse = lisa.cross_attention(q, k, k, bias=bias, return_lse=True)
        assert out.shape == q.shape and lse.shape == (0, 2, 5)
        dq, dk, dv, dtable = lisa.cross_attention_backward(q, k, k, out, lse, out, bias=bias)
        assert dq.shape == q.shape and dk.shape == k.shape and not dtable.any() and torch.isfinite(dtable).all()


# ------------------------------------------------------------------ scores far from 0

class Far(Case):
    """Scores 2^exponent r_i k_j with whole r_i, k_j of 8 bits: exact in fp32, in every order. One key of a row stands at
    least 2^exponent 128 above the rest (2^12 and more), whose weights are 0 in any precision: o is that key's value and lse
    its score."""

    def __init__(self, lisa, dtype, n, m, exponent, *, bias=None, signs="both"):
        super().__init__(lisa, dtype, 2, 2, 2, n, m, 64, bias=bias, scale=1.0)
        g = torch.Generator().manual_seed(exponent)
        r = torch.randint(128, 256, (2, 2, n), generator=g) * (2 * torch.randint(0, 2, (2, 2, n), generator=g) - 1)
        w = torch.randint(-100, 100, (2, 2, m), generator=g)
        top = torch.stack([torch.randperm(m, generator=g)[:2] for _ in range(4)]).view(2, 2, 2)
        w.scatter_(2, top, torch.tensor([127, -127]).expand(2, 2, 2))
        if signs == "negative":     # every score of a row below 0
            r, w = -r.abs(), w + 128
        self.q_ref, self.k_ref = torch.zeros_like(self.q_ref), torch.zeros_like(self.k_ref)
        self.q_ref[..., 5], self.k_ref[..., 5] = (r * 2.0 ** exponent).to(dtype), w.to(dtype)
        assert torch.equal(self.q_ref[..., 5].double(), r.double() * 2.0 ** exponent)
        self.q.copy_(self.q_ref)
        self.k.copy_(self.k_ref)
        self.s = self.q_ref.double() @ self.k_ref.double().transpose(-1, -2)
        self.best = self.s.argmax(-1)
        if bias is not None:
            self.s += self.table.double().t()[:, self.index]


@pytest.mark.parametrize("signs", ["both", "negative"])
@pytest.mark.parametrize("exponent", [5, 15, 20, 26, 60, 100])
@pytest.mark.parametrize("dtype,n,m,bias", [(BF16, 150, 300, None), (BF16, 150, 1100, None), (BF16, 300, 90, None),
                                            (BF16, 150, 1100, LOG), (BF16, 150, 300, NEAR), (BF16, 1, 700, None),
                                            (BF16, 3, 700, LOG), (F32, 70, 300, None), (F32, 70, 300, LOG)])
def test_finite_scores_of_any_size(lisa, dtype, n, m, bias, exponent, signs):
    """Up to 2^116: the outputs stay those of a softmax. lse is off by the roundings of log2(e) times the scale, of the
    score, of its product with ln 2 and of ln 2 itself, 2^-24 each, and one in fp32 beside them; the other keys' part of it
    (below 2^-4000) and log2 of a sum of 1 are nothing."""
    c = Far(lisa, dtype, n, m, exponent, bias=bias, signs=signs)
    out, lse = c.forward()
    value = c.v_ref.gather(2, c.best[..., None].expand(-1, -1, -1, 64))
    # its weight may stand at another power of two than 1 and is rounded for the product, the result once more
    off = 2.02 * 2.0 ** -8 if dtype == BF16 else 4 * 2.0 ** -24
    assert ((out.double().cpu() - value.double()).abs() <= off * value.double().abs()).all()
    want = c.s.amax(-1)
    assert ((lse.double().cpu() - want).abs() <= 5.1 * 2.0 ** -24 * (want.abs() + 8)).all()
    if n > 1 and exponent >= 15:     # |lse| > 2^20: no gradient
        assert not any(x.any() for x in c.backward(out, lse))


# ------------------------------------------------------------------ grids wider than a tile

WIDE = [((2, 200), (2, 200), ("exact", 199)), ((3, 130), (1, 129), ("exact", 129)), ((2, 300), (3, 150), ("exact", 40)),
        ((2, 200), (2, 150), ("log", 32, 128)), ((1, 1), (2, 500), ("log", 32, 128)), ((3, 2), (5, 380), ("exact", 379)),
        ((2, 400), (2, 700), ("exact", 699))]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("q,k,cols", WIDE)
def test_bias_gradient_of_grids_wider_than_a_tile(lisa, dtype, q, k, cols):
    """Whole numbers 1 to 8: sums below 2^24, so exact, and one pair too few or too many shows."""
    b, table, index = _matrix(lisa, q, k, {"rows": ("exact", max(q[0], k[0]) - 1), "cols": cols})
    x = torch.randint(1, 9, (3, b.n, b.m), generator=torch.Generator().manual_seed(7))
    want = torch.zeros(table.shape, dtype=torch.int64)
    for h in range(3):
        want[:, h].index_add_(0, index.reshape(-1), x[h].reshape(-1))
    assert want.max() < 1 << 24
    assert torch.equal(lisa.relative_bias_backward(b, x.to(dtype).cuda()).cpu().long(), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("q,k,cols", [WIDE[0], WIDE[3], WIDE[5], WIDE[6]])
def test_attention_on_grids_wider_than_a_tile(lisa, dtype, q, k, cols):
    Case(lisa, dtype, 2, 2, 1, q, k, 64, bias={"rows": ("exact", max(q[0], k[0]) - 1), "cols": cols}).check()


@pytest.mark.parametrize("q,k,how", [((1, 1), (127, 129), None), ((1, 1), (16384, 1), ("exact", 50)),
                                     ((1, 32), (2, 8161), None)])
def test_every_grid_of_the_most_offsets_launches(lisa, q, k, how):
    """16383 and 16384 offsets with 16322 to 16384 keys: offsets and key offsets at their largest at once."""
    bias = _grid(q, k) if how is None else {"rows": how, "cols": ("exact", 0)}
    Case(lisa, BF16, 1, 1, 1, q, k, 64, bias=bias).check()


# ------------------------------------------------------------------ long sums

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("q,k,how", MATRICES)
def test_bias_matrix_gradient_misses_no_pair(lisa, dtype, q, k, how):
    """Whole numbers 1 to 8, exact in either type, whose sums stay below 2^24: every partial sum is exact in fp32, so the
    gradient is the exact sum, and one pair too few or too many shows."""
    b, table, index = _matrix(lisa, q, k, how)
    x = torch.randint(1, 9, (3, b.n, b.m), generator=torch.Generator().manual_seed(6))
    want = torch.zeros(table.shape, dtype=torch.int64)
    for h in range(3):
        want[:, h].index_add_(0, index.reshape(-1), x[h].reshape(-1))
    assert want.max() < 1 << 24
    assert torch.equal(lisa.relative_bias_backward(b, x.to(dtype).cuda()).cpu().long(), want)


@pytest.mark.parametrize("step", [1, 1 << 23])
def test_bias_matrix_gradient_of_the_most_queries(lisa, step):
    """2^22 x 2 pairs, of 1 and 2: sums below 2^24, exact."""
    n = 1 << 22
    b = lisa.RelativeBias(torch.zeros(3, 1, device="cuda"), (1, n), (1, 2), cols=lisa.exact_buckets(1), key_step=(1, step))
    x = torch.randint(1, 3, (1, n, 2), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda")
    offset = step * torch.arange(2, device="cuda") - torch.arange(n, device="cuda")[:, None]
    want = torch.zeros(3, dtype=torch.int64, device="cuda")
    want.index_add_(0, (offset.clamp(-1, 1) + 1).reshape(-1), x.reshape(-1))
    assert want.max() < 1 << 24
    assert torch.equal(lisa.relative_bias_backward(b, x.float())[:, 0].long(), want)


def test_the_most_queries_with_sums_that_add_up(lisa):
    """2^22 queries of two keys, fp32, one key in the bucket before the query and one in the bucket behind it, and dO along
    v_1 - v_0: every dS of a key has the same sign, so each sum is as large as its terms together.

    A term's error, in units of 2^-24: a weight's score has 18 roundings of sum |q k| / 4 <= 32, 576 for each of the two
    weights, lse 32 each, exp 40 each, and dP, delta and their difference 18 each of |dO| |v|, at most 8 times
    dP_1 - dP_0 here: 2048 units of dS hold all of it.
    A bucket's sum: runs of 128 in a tile, 1024 of the tiles, 32 of those, so at most 1184 further units of the sum.
    dK and dV add n terms one by one: each addition is off by at most 2^-24 of the sum so far, one way or the other, which
    comes to sqrt(n / 3) units rms; 8 sqrt(n) is taken."""
    n, d = 1 << 22, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    q = 1 + torch.randn(1, 1, n, d, generator=g, device="cuda")
    k, v = (torch.randn(1, 1, 2, d, generator=g, device="cuda") for _ in range(2))
    do = (0.5 + torch.rand(1, 1, n, 1, generator=g, device="cuda")) * (v[:, :, 1:] - v[:, :, :1])
    table = torch.randn(3, 1, generator=g, device="cuda")
    bias = lisa.RelativeBias(table, (1, n), (1, 2), cols=lisa.exact_buckets(1), key_step=(1, 1 << 23), query_start=(0, 1))
    out, lse = lisa.cross_attention(q, k, v, bias=bias, return_lse=True)
    dq, dk, dv, dtable = lisa.cross_attention_backward(q, k, v, out, lse, do, bias=bias)
    Q, K, V, G = (x[0, 0].double() for x in (q, k, v, do))
    s = Q @ K.t() / 4 + table.double()[[0, 2], 0]
    assert (Q.abs() @ K.abs().t() / 4).max() <= 32
    p = torch.softmax(s, -1)
    dp = G @ V.t()
    size = G.norm(dim=1, keepdim=True) * V.norm(dim=1)
    assert (size.amax(1) <= 8 * (dp[:, 1] - dp[:, 0])).all()
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    assert (ds[:, 1] > 0).all() and (ds[:, 0] < 0).all()
    unit, run = 2.0 ** -24, 8 * n ** 0.5
    most = ds.abs().amax(1, keepdim=True)
    term = 2048 * unit * most
    want = torch.stack((ds[:, 0].sum(), ds[:, 1].sum()))
    bound = term.sum() + 1184 * unit * want.abs()
    assert (bound <= 3e-4 * want.abs()).all()
    assert ((dtable[[0, 2], 0].double() - want).abs() <= bound).all() and dtable[1, 0] == 0
    assert ((dq[0, 0].double() - ds @ K / 4).abs() <= (term * 2 + 4 * unit * most) @ K.abs().amax(0, keepdim=True) / 4).all()
    off = (term.sum() + run * unit * ds.abs().sum(0))[:, None]
    mag = Q.abs().amax() / 4
    want_k = ds.t() @ Q / 4
    assert ((dk[0, 0].double() - want_k).abs() <= off * mag).all() and (off * mag <= 0.05 * want_k.abs()).all()
    want_v = p.t() @ G
    # the error of p: less than that of dS, which holds both weights' and dP's
    assert ((dv[0, 0].double() - want_v).abs() <= (2048 + run) * unit * (p.t() @ G.abs())).all()
    assert ((2048 + run) * unit * (p.t() @ G.abs()) <= 2e-3 * want_v.abs()).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", [0.0, 3e5, -3e5, -1e9, 2.0 ** 40, "bias"])
@pytest.mark.parametrize("n", [1, 150])
def test_equal_scores_of_any_size_weigh_every_key_alike(lisa, dtype, score, n):
    """Every key has the same score, of any size: o is the mean of the valid values, whatever parts the keys are taken in.
    Weights of one size are exact up to a common factor that p's rounding may miss by half a step; the rest is the
    sums' and the result's rounding."""
    lens = [1100, 129, 257, 1000, 0, 513]
    c = Case(lisa, dtype, 6, 2, 2, n, 1100, 64, lens=lens, scale=1.0, garbage=True,
             bias={"cols": ("exact", 0)} if score == "bias" else None)
    if score == "bias":     # -1e9 for every pair: nothing of the scores (below 128 / 64 units) is left beside it in fp32
        c.q.mul_(0.25)
        c.bias.table.fill_(-1e9)
        score = -1e9
    else:
        c.q.zero_()
        c.q[..., 0] = score
        c.k[..., 0] = 1.0
        score = float(c.q[0, 0, 0, 0])
    out, lse = c.forward()
    for b, L in enumerate(lens):
        if L == 0:
            assert not out[b].any() and (lse[b] == -math.inf).all()
            continue
        v = c.v_ref[b, :, :L].double()
        r = ref.R[dtype]
        bound = 2.02 * r * v.mean(1).abs() + (L + 8) * ref.U[dtype] * v.abs().mean(1)
        assert ((out[b].double().cpu() - v.mean(1)[:, None]).abs() <= bound[:, None]).all(), L
        want = score + math.log(L)
        assert ((lse[b].double() - want).abs() <= 5.1 * 2.0 ** -24 * (abs(score) + 8) + (L + 8) * ref.U[dtype] + 8 * ref.EX2).all()


def test_long_sums_over_queries_and_heads_fp32(lisa):
    """One key, so every weight is exactly 1 and dV is the sum of dO over 16384 queries of 4 heads: 65536 terms of
    1025 units of 2^-10.  A tile's 64 terms add up exactly (65600 units); the 1024 tiles are off by at most 2^-24 of the sum
    each.  Term by term the sum would lose a unit with every addition past 2^24 units, 7e-4 of it in all."""
    n, heads, d = 16384, 4, 64
    q, k = torch.randn(1, heads, n, d, device="cuda"), torch.randn(1, 1, 1, d, device="cuda")
    dout = torch.full_like(q, 1 + 2.0 ** -10)
    out, lse = lisa.cross_attention(q, k, k, return_lse=True)
    dv = lisa.cross_attention_backward(q, k, k, out, lse, dout)[2]
    want = n * heads * (1 + 2.0 ** -10)
    assert ((dv.double() - want).abs() <= 1024 * 2.0 ** -24 * want).all()


@pytest.mark.parametrize("n", [1, 70])
def test_long_sums_over_keys_fp32(lisa, n):
    """65536 keys of one score: unscaled weights of exactly 1, values of 1025 units of 2^-10, so o is 1025 units as well.
    A tile's 64 terms add up exactly; the 1024 tiles are off by at most 2^-24 of the sum each, the division and the result
    by 2^-24 each.  Term by term the sum would be 7e-4 off."""
    m = 1 << 16
    q, k = torch.zeros(1, 1, n, 16, device="cuda"), torch.randn(1, 1, m, 16, device="cuda")
    v = torch.full_like(k, 1 + 2.0 ** -10)
    out, lse = lisa.cross_attention(q, k, v, return_lse=True)
    assert ((out.double() - (1 + 2.0 ** -10)).abs() <= 1027 * 2.0 ** -24 * (1 + 2.0 ** -10)).all()
    assert ((lse.double() - math.log(m)).abs() <= 4 * 2.0 ** -24 * math.log(m)).all()
