"""The 64-bit restatement of the cross attention against central differences of
its own forward, and the bucket rule against values worked by hand (CPU)."""
import math

import pytest
import torch

import attention_ref as ref


def test_log_buckets_by_hand():
    rule = ("log", 32, 128)     # E = 8; far borders at 8 * 16^(t / 8): 8, 11.3, 16, 22.6, 32, 45.3, 64, 90.5
    want = {0: 0, -1: 1, -7: 7, -8: 8, -11: 8, -12: 9, -15: 9, -16: 10, -22: 10, -23: 11, -31: 11, -32: 12, -45: 12,
            -46: 13, -63: 13, -64: 14, -90: 14, -91: 15, -127: 15, -128: 15, -5000: 15, 1: 17, 7: 23, 8: 24, 16: 26,
            64: 30, 128: 31, 9999: 31}
    for x, b in want.items():
        assert ref.bucket_of(x, rule) == b, x
    assert [ref.bucket_of(x, ("exact", 2)) for x in (-9, -2, -1, 0, 1, 2, 7)] == [0, 0, 1, 2, 3, 4, 4]
    assert [ref.bucket_of(x, ("log", 4, 2)) for x in (-5, -1, 0, 1, 2)] == [1, 1, 0, 3, 3]


@pytest.mark.parametrize("lens", [None, [3, 0]])
def test_gradients_against_differences(lens):
    g = torch.Generator().manual_seed(5)
    B, h, kv, n, m, d = 2, 4, 2, 5, 7, 3
    q, k, v, do = (torch.randn(*s, generator=g, dtype=torch.float64)
                   for s in ((B, h, n, d), (B, kv, m, d), (B, kv, m, d), (B, h, n, d)))
    rule = ("log", 8, 5)
    table = torch.randn(8, h, generator=g, dtype=torch.float64)
    index = ref.bucket_index((1, n), (1, m), ("exact", 0), rule)
    kw = dict(scale=0.6, lens=lens, index=index)
    r = ref.attention(q, k, v, do, table=table, **kw)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dtable", table)):
        dirn = torch.randn(x.shape, generator=g, dtype=torch.float64)
        step = 1e-5
        vals = []
        for sign in (1, -1):
            args = {"dq": q, "dk": k, "dv": v, "dtable": table}
            args[name] = x + sign * step * dirn
            o = ref.attention(args["dq"], args["dk"], args["dv"], table=args["dtable"], **kw)["o"][0]
            vals.append(float((o * do).sum()))
        want = (vals[0] - vals[1]) / (2 * step)
        got = float((r[name][0] * dirn).sum())
        assert math.isclose(got, want, rel_tol=1e-7, abs_tol=1e-8), name
