"""The cross attention's and the relative bias's C ABI on the host: refusals
and sizes, decided before anything is launched (no GPU)."""
import math

import pytest
import torch

from hop_stochastic_vision_gb300 import attention as att
from hop_stochastic_vision_gb300 import build as lisa_build
from hop_stochastic_vision_gb300 import lisa

FAKE = 1 << 20          # 16-byte aligned, never dereferenced
OK, INV, UNS, WSP = lisa.LISA_OK, lisa.LISA_ERR_INVALID_ARG, lisa.LISA_ERR_UNSUPPORTED, lisa.LISA_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def built():
    lisa_build.build()
    lisa.load()


def _bias(q_grid=(1, 8), k_grid=(1, 8), rows=None, cols=None, step=(1, 1), start=(0, 0), starts=None, table=None):
    rows = att.exact_buckets(0) if rows is None else rows
    cols = att.log_buckets(32, 128) if cols is None else cols
    return att.lisa_rel_bias(FAKE + (64 << 20) if table is None else table, *q_grid, *k_grid, *step, *start, starts,
                             rows, cols)


def _strides(h, t, d, **over):
    return att.lisa_strides(over.get("batch", h * t * d), over.get("head", t * d), over.get("token", d))


def _forward(**over):
    a = dict(Q=FAKE, K=FAKE + (1 << 20), V=FAKE + (2 << 20), O=FAKE + (3 << 20), lse=FAKE + (4 << 20), B=2, heads=4,
             kv_heads=2, n=8, m=8, d=16, scale=0.25, kv_lens=None, bias=None, dtype=lisa.LISA_F32,
             ws=FAKE + (32 << 20), wbytes=1 << 40)
    a.update(over)
    qs = a.get("qs", _strides(a["heads"], a["n"], a["d"]))
    ks = a.get("ks", _strides(a["kv_heads"], a["m"], a["d"]))
    return att.lisa_cross_attention(a["Q"], qs, a["K"], ks, a["V"], a.get("vs", ks), a["O"], a.get("os", qs), a["lse"],
                                    a["B"], a["heads"], a["kv_heads"], a["n"], a["m"], a["d"], a["scale"],
                                    a["kv_lens"], a["bias"], a["dtype"], a["ws"], a["wbytes"], 0)


BAD = [
    (dict(Q=0), INV), (dict(K=0), INV), (dict(V=0), INV),
    (dict(Q=FAKE + 8), INV), (dict(V=FAKE + (2 << 20) + 4), INV),
    (dict(B=-1), INV), (dict(n=-1), INV), (dict(m=-1), INV), (dict(heads=3), INV), (dict(kv_heads=0), INV),
    (dict(d=0), INV), (dict(d=48), UNS), (dict(d=128), UNS), (dict(dtype=2), INV),
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
    (dict(kv_lens=FAKE + 2), INV), (dict(B=70000), UNS), (dict(n=(1 << 22) + 1), UNS),
    (dict(qs=None), INV), (dict(ks=None), INV),
    (dict(qs=_strides(4, 8, 16, token=18)), INV),      # not a multiple of 16 bytes
    (dict(qs=_strides(4, 8, 16, token=12)), INV),      # tokens overlap
    (dict(ks=_strides(2, 8, 16, head=-128)), INV),
    (dict(bias=_bias(q_grid=(1, 9))), INV),            # another n
    (dict(bias=_bias(k_grid=(2, 8))), INV),
    (dict(bias=_bias(table=0)), INV), (dict(bias=_bias(table=FAKE + 2)), INV),
    (dict(bias=_bias(step=(0, 1))), INV),
    (dict(bias=_bias(cols=att.lisa_axis_rule(2, 5, 2))), INV),
    (dict(bias=_bias(cols=att.lisa_axis_rule(0, 4, 2))), INV),
    (dict(bias=_bias(cols=att.exact_buckets(8192))), UNS),
    (dict(bias=_bias(cols=att.log_buckets(30, 128))), INV), (dict(bias=_bias(cols=att.log_buckets(32, 8))), INV),
    (dict(bias=_bias(cols=att.log_buckets(132, 900))), UNS),
    (dict(bias=_bias(q_grid=(2, 4), starts=FAKE)), INV),   # own starts: sequences only
]


@pytest.mark.parametrize("over,status", BAD + [
    (dict(O=0), INV), (dict(O=FAKE + (3 << 20) + 8), INV), (dict(lse=FAKE + 1), INV),
    (dict(O=FAKE), INV), (dict(O=FAKE + (1 << 20) + 256), INV),         # overlaps Q, K
    (dict(os=_strides(4, 8, 16, batch=0)), INV),                        # an output entry repeated
    (dict(os=_strides(4, 8, 16, head=16)), INV),                        # heads and tokens in one place
    (dict(os=att.lisa_strides(8 * 64, 16, 60)), INV), (dict(os=att.lisa_strides(7 * 64, 16, 64)), INV),
    (dict(lse=FAKE + 64), INV), (dict(lse=FAKE + (3 << 20) + 64), INV), (dict(O=FAKE + (64 << 20), bias=_bias()), INV),
    (dict(B=60000, heads=60000, kv_heads=60000), UNS),
])
def test_forward_rejects_before_launch(over, status):
    assert _forward(**over) == status


def _backward(**over):
    a = dict(Q=FAKE, K=FAKE + (1 << 20), V=FAKE + (2 << 20), O=FAKE + (3 << 20), lse=FAKE + (4 << 20),
             dO=FAKE + (5 << 20), dQ=FAKE + (6 << 20), dK=FAKE + (7 << 20), dV=FAKE + (8 << 20), dtable=None, B=2,
             heads=4, kv_heads=2, n=8, m=8, d=16, scale=0.25, kv_lens=None, bias=None, dtype=lisa.LISA_F32,
             ws=FAKE + (32 << 20), wbytes=1 << 40)
    a.update(over)
    if a["bias"] is not None and "dtable" not in over:
        a["dtable"] = FAKE + (9 << 20)
    qs = a.get("qs", _strides(a["heads"], a["n"], a["d"]))
    ks = a.get("ks", _strides(a["kv_heads"], a["m"], a["d"]))
    return att.lisa_cross_attention_backward(
        a["Q"], qs, a["K"], ks, a["V"], a.get("vs", ks), a["O"], a.get("os", qs), a["lse"], a["dO"], a.get("dos", qs),
        a["dQ"], a["dK"], a["dV"], a["dtable"], a["B"], a["heads"], a["kv_heads"], a["n"], a["m"], a["d"], a["scale"],
        a["kv_lens"], a["bias"], a["dtype"], a["ws"], a["wbytes"], 0)


@pytest.mark.parametrize("over,status", BAD + [
    (dict(O=0), INV), (dict(lse=0), INV), (dict(dO=0), INV), (dict(dQ=0), INV), (dict(dK=0), INV), (dict(dV=0), INV),
    (dict(dQ=FAKE + (6 << 20) + 8), INV), (dict(dO=FAKE + (5 << 20) + 8), INV), (dict(lse=FAKE + 2), INV),
    (dict(dQ=FAKE + (7 << 20)), INV), (dict(dK=FAKE + (1 << 20)), INV), (dict(dV=FAKE + (4 << 20)), INV),
    (dict(dtable=FAKE + (9 << 20)), INV),                               # without a bias
    (dict(bias=_bias(), dtable=None), INV), (dict(bias=_bias(), dtable=FAKE + (6 << 20)), INV),
    (dict(bias=_bias(starts=FAKE)), INV),                               # forward only
    (dict(dos=_strides(4, 8, 16, token=10)), INV),
    (dict(ws=0), WSP), (dict(wbytes=16), WSP), (dict(ws=FAKE + (32 << 20) + 8), INV),
])
def test_backward_rejects_before_launch(over, status):
    assert _backward(**over) == status


def test_empty_problems_launch_nothing():
    assert _forward(B=0, Q=0, K=0, V=0, O=0, lse=0) == OK
    assert _forward(n=0, Q=0, K=0, V=0, O=0, lse=0) == OK
    assert _forward(heads=0, kv_heads=0, Q=0, K=0, V=0, O=0, lse=0) == OK
    assert _backward(B=0, Q=0, K=0, V=0, O=0, dO=0, dQ=0, dK=0, dV=0, ws=0) == OK
    assert _backward(n=0, m=0, Q=0, K=0, V=0, O=0, dO=0, dQ=0, dK=0, dV=0, ws=0) == OK


def test_workspace_bytes():
    ws = att.lisa_cross_attention_backward_workspace_bytes
    plain = ws(2, 4, 2, 8, 8, 16, None, lisa.LISA_F32)
    assert plain >= 2 * 4 * 8 * 4
    assert ws(2, 4, 2, 8, 8, 16, _bias(), lisa.LISA_F32) > plain
    assert ws(2, 4, 3, 8, 8, 16, None, lisa.LISA_F32) == 0 and ws(2, 4, 2, 8, 8, 48, None, lisa.LISA_F32) == 0
    assert ws(0, 4, 2, 8, 8, 16, None, lisa.LISA_F32) == 0
    ws = att.lisa_cross_attention_workspace_bytes
    assert ws(2, 4, 3, 8, 8, 16, None, lisa.LISA_F32) == 0                     # heads not shared evenly
    assert ws(2, 4, 2, 8, 8, 16, None, lisa.LISA_F32) == 0                     # nothing needed
    plain = ws(2, 4, 2, 200, 8, 16, None, lisa.LISA_BF16)
    assert plain > 0 and ws(2, 4, 2, 200, 8, 16, _bias((1, 200)), lisa.LISA_BF16) > plain
    assert ws(2, 4, 2, 1, 800, 16, None, lisa.LISA_BF16) == 0                  # single tokens
    assert ws(2, 4, 2, 200, 8, 16, _bias((1, 200), step=(1, 0)), lisa.LISA_BF16) == 0
    assert att.lisa_relative_bias_backward_workspace_bytes(_bias(), 4) > 0
    assert att.lisa_relative_bias_backward_workspace_bytes(_bias(step=(1, 0)), 4) == 0


@pytest.mark.parametrize("over,status", [
    (dict(q_grid=(0, 8)), INV), (dict(step=(1, 0)), INV), (dict(starts=FAKE), INV), (dict(table=0), INV),
    (dict(cols=att.exact_buckets(-1)), INV), (dict(rows=att.lisa_axis_rule(7, 1, 0)), INV),
    (dict(q_grid=(65, 65), k_grid=(65, 65), rows=att.exact_buckets(64), cols=att.exact_buckets(64)), UNS),
    (dict(start=(0, 1 << 30)), UNS), (dict(q_grid=(1, 1 << 20), k_grid=(1, 1 << 20)), UNS),
])
def test_bias_matrix_rejects_before_launch(over, status):
    b = _bias(**over)
    assert att.lisa_relative_bias(b, 4, FAKE, lisa.LISA_F32, 0) == status
    if "table" not in over:   # the gradient does not read the table
        assert att.lisa_relative_bias_backward(b, 4, FAKE, lisa.LISA_F32, FAKE + (1 << 24), FAKE + (2 << 24), 1 << 40,
                                               0) == status


def test_bias_matrix_rejects_other_arguments():
    b = _bias()
    assert att.lisa_relative_bias(None, 4, FAKE, lisa.LISA_F32, 0) == INV
    assert att.lisa_relative_bias(b, 0, FAKE, lisa.LISA_F32, 0) == INV
    assert att.lisa_relative_bias(b, 4, 0, lisa.LISA_F32, 0) == INV
    assert att.lisa_relative_bias(b, 4, FAKE + 8, lisa.LISA_F32, 0) == INV
    assert att.lisa_relative_bias(b, 4, FAKE, 3, 0) == INV
    assert att.lisa_relative_bias(b, 4, FAKE + (64 << 20), lisa.LISA_F32, 0) == INV        # over the table
    grad = att.lisa_relative_bias_backward
    assert grad(b, 4, FAKE, lisa.LISA_F32, FAKE, FAKE + (2 << 24), 1 << 40, 0) == INV      # dtable over dbias
    assert grad(b, 4, FAKE, lisa.LISA_F32, FAKE + (1 << 24), 0, 1 << 40, 0) == WSP
    assert grad(b, 4, FAKE, lisa.LISA_F32, FAKE + (1 << 24), FAKE + (2 << 24), 8, 0) == WSP
    assert grad(b, 4, FAKE, lisa.LISA_F32, FAKE + (1 << 24), FAKE + (2 << 24) + 4, 1 << 40, 0) == INV
    # a grid of 64 x 64 on both sides fits
    big = _bias(q_grid=(64, 64), k_grid=(64, 64), rows=att.exact_buckets(63), cols=att.exact_buckets(63))
    assert att.lisa_relative_bias_backward_workspace_bytes(big, 4) > 0


def test_tensor_calls_refuse_what_is_not_on_a_gpu():
    x = torch.zeros(1, 1, 4, 16)
    with pytest.raises(ValueError):
        lisa.cross_attention(x, x, x)
    with pytest.raises(ValueError):
        lisa.cross_attention_backward(x, x, x, x, torch.zeros(1, 1, 4), x)
    with pytest.raises(ValueError):
        lisa.cross_attention(x.half(), x.half(), x.half())
    with pytest.raises(ValueError):
        lisa.RelativeBias(torch.zeros(32, 4), (1, 4), (1, 4), cols=lisa.log_buckets(32, 128))


# ------------------------------------------------------------------ a bias whose tensors change between calls

class OnGpu(torch.Tensor):
    """A tensor of the host that calls itself one of cuda:0, for checks that launch nothing."""
    is_cuda = True
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


def _on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def _tokens(starts):
    return lisa.RelativeBias(_on_gpu(32, 4), (1, 1), (1, 9), cols=lisa.log_buckets(32, 128), query_start=starts)


BAD_STARTS = {"int64": lambda: _on_gpu(6, dtype=torch.int64), "host": lambda: torch.zeros(6, dtype=torch.int32),
              "strided": lambda: _on_gpu(12, dtype=torch.int32)[::2], "matrix": lambda: _on_gpu(6, 1, dtype=torch.int32)}


@pytest.mark.parametrize("what", BAD_STARTS)
def test_starts_are_checked_whenever_they_are_used(what):
    with pytest.raises(ValueError):
        _tokens(BAD_STARTS[what]())
    b = _tokens(_on_gpu(6, dtype=torch.int32))
    b.starts = BAD_STARTS[what]()
    with pytest.raises(ValueError):
        b.current()
    good = b.starts = _on_gpu(7, dtype=torch.int32)
    assert b.current().starts == good.data_ptr()
    b.starts = None
    assert b.current().starts is None


SAME_PLACE = {"fewer rows": lambda t: t[:20], "transposed": lambda t: t.t(), "one dimension": lambda t: t.view(-1),
              "other type": lambda t: t.view(torch.int32), "other shape": lambda t: t.view(4, 32),
              "fewer heads": lambda t: t[:, :3], "host": lambda t: t.as_subclass(torch.Tensor)}


@pytest.mark.parametrize("how", SAME_PLACE)
def test_the_table_is_checked_whenever_it_is_used(how):
    """Another tensor at the same address is another table."""
    table = _on_gpu(32, 4)
    b = lisa.RelativeBias(table, (1, 5), (1, 9), cols=lisa.log_buckets(32, 128))
    b.table = SAME_PLACE[how](table)
    assert b.table.data_ptr() == table.data_ptr()
    for use in (b.current, lambda: lisa.relative_bias(b), lambda: lisa.relative_bias_backward(b, table)):
        with pytest.raises(ValueError):
            use()
    b.table = table
    assert b.current().table == table.data_ptr()


@pytest.mark.parametrize("q,k", [((2, 200), (2, 200)), ((3, 130), (1, 129)), ((1, 1), (127, 129)), ((2, 1), (2, 300)),
                                 ((3, 2), (5, 380))])
@pytest.mark.parametrize("rule", ["exact", "log"])
def test_the_gradients_workspace_holds_what_a_tile_of_a_wide_grid_spans(q, k, rule):
    """128 tokens that cross the end of a row stand in all columns of a grid, however many those are."""
    n, m = q[0] * q[1], k[0] * k[1]

    def spans(count, cols):        # per tile: the rows and the columns of its tokens
        tiles = [[(t // cols, t % cols) for t in range(t0, min(t0 + 128, count))] for t0 in range(0, count, 128)]
        return [(max(r) - min(r), max(c) - min(c)) for r, c in (zip(*t) for t in tiles)]

    cols = att.exact_buckets(max(q[1], k[1]) - 1) if rule == "exact" else att.log_buckets(32, 128)
    rows = att.exact_buckets(max(q[0], k[0]) - 1)
    most = max((a[0] + b[0] + 1) * (min(a[1] + b[1] + 1, cols.buckets) if rule == "exact" else 32)
               for a in spans(n, q[1]) for b in spans(m, k[1]))
    tiles = -(-n // 128) * -(-m // 128)
    assert att.lisa_relative_bias_backward_workspace_bytes(_bias(q, k, rows, cols), 3) >= 3 * tiles * most * 4


BEYOND = 1 << 32       # times anything: 0 in 32 bits


@pytest.mark.parametrize("which", ["queries", "keys", "batch", "heads"])
def test_sizes_beyond_32_bits_are_refused(which):
    many = {"queries": (1, 1, BEYOND + 1, 16), "keys": (1, 1, 1, 16), "batch": (BEYOND + 1, 1, 1, 16),
            "heads": (1, BEYOND + 1, 1, 16)}[which]
    q = _on_gpu(1, 1, 1, 16).expand(*many)
    k = {"queries": _on_gpu(1, 1, 1, 16), "keys": _on_gpu(1, 1, 1, 16).expand(1, 1, BEYOND + 1, 16)}.get(which, q)
    for call in (lambda: lisa.cross_attention(q, k, k, out=q),
                 lambda: lisa.cross_attention_backward(q, k, k, q, _on_gpu(1).expand(q.shape[:3]), q)):
        with pytest.raises(lisa.LisaError) as e:
            call()
        assert e.value.status == UNS


@pytest.mark.parametrize("over", [dict(q_grid=(1, BEYOND + 5)), dict(k_grid=(BEYOND + 1, 9)), dict(key_step=(1, BEYOND + 1)),
                                  dict(query_start=(0, BEYOND)), dict(query_start=(-BEYOND - 1, 0))])
def test_positions_beyond_32_bits_are_refused(over):
    args = {**dict(q_grid=(1, 5), k_grid=(1, 9), cols=lisa.log_buckets(32, 128)), **over}
    with pytest.raises(ValueError):
        lisa.RelativeBias(_on_gpu(32, 4), **args)


def test_bucket_rules_beyond_32_bits_are_refused():
    for call in (lambda: lisa.exact_buckets(BEYOND), lambda: lisa.exact_buckets(1 << 30),
                 lambda: lisa.log_buckets(BEYOND + 32, 128), lambda: lisa.log_buckets(32, BEYOND + 128)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("over", [dict(O=FAKE + (80 << 20)), dict(lse=FAKE + (80 << 20) - 64)])
def test_outputs_over_the_starts_are_refused(over):
    b = _bias(starts=FAKE + (80 << 20))
    assert _forward(bias=b, **over) == INV


@pytest.mark.parametrize("over", [
    dict(m=0, dQ=FAKE), dict(m=0, dQ=FAKE + (3 << 20)), dict(m=0, dQ=FAKE + (4 << 20)), dict(m=0, dQ=FAKE + (5 << 20)),
    dict(m=0, dQ=FAKE + (6 << 20) + 8), dict(m=0, dQ=FAKE + (9 << 20), bias=_bias()),
    dict(m=0, dQ=FAKE + (64 << 20), bias=_bias()), dict(n=0, dK=FAKE + (1 << 20)), dict(n=0, dV=FAKE + (1 << 20) + 64),
    dict(n=0, dV=FAKE + (7 << 20)), dict(n=0, dK=FAKE + (7 << 20) + 4)])
def test_empty_problems_zero_no_input_and_no_output_twice(over):
    assert _backward(**over) == INV


def test_empty_problems_take_the_rules_that_the_others_take():
    assert _backward(m=0, bias=_bias(cols=att.exact_buckets(8192))) == UNS
    assert _backward(m=0, bias=_bias(cols=att.lisa_axis_rule(0, 4, 2))) == INV
