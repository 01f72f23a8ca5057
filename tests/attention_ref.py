"""The cross attention and the relative position bias from their definition, in
64 bits on the CPU, with elementwise bounds of what a kernel of a given data
type may be off by.

Bounds.  u is the rounding of one operation in the kernels' accumulation: 2^-24
for fp32 arithmetic; 2^-22 where sums run on the tensor cores or through the
special-function unit's 2^x (both may drop the last bits instead of rounding
them).  r is the rounding of an operand or a result to the data type: at most
half a step, 2^-8 for bf16 (finfo.eps / 2), 2^-24 for fp32.  With N the number
of terms, a sum's error is at most N u sum|terms|; the products of rounded
operands add r per rounded operand.  Every bound below is that first-order sum,
taken 1.05 times for the second order.

  s     Es = u (d + 8) (scale |q|.|k| + |b|)
  p     Ep = p (Es + max_j Es + u (m + 8) + 8 u |s - lse|) + f
        f = 2^-126: 2^x (and a product) below the smallest normal fp32 number is
        flushed to 0, an error of up to f in p whatever p is; through dP, q and k
        it reaches the gradients times their size (some hundreds here) and n terms
  o     Eo = sum_j (Ep + (r + m u) p) |v| + r |o|
  dP    u (d + 2) |dO|.|v|
  dS    EdS = Ep |dP - delta| + p (EdP + Edelta + 4 u (|dP| + |delta|)) + f
        Edelta = |dO|.Eo + u (d + 2) |dO|.|o|   (delta from the rounded output)
        or, where it is summed in fp32, sum_j (Ep + m u p) |dP| + p EdP
  dQ    scale sum_j (EdS + (r + m u) |dS|) |k| + r |dQ|      dK likewise over i
  dV    sum_i (Ep + (r + n u) p) |dO| + r |dV|
  table the summed EdS, unrounded, + 64 u sum |p| (|dP| + |delta|)
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -22}
R = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F = 2.0 ** -126       # smallest normal fp32 number
EX2 = 2.0 ** -22      # relative error of the special-function unit's 2^x, in either data type


def bucket_of(x, rule):
    """Bucket of one offset, rule = ("exact", D) or ("log", buckets, D); whole numbers only."""
    if rule[0] == "exact":
        return min(max(x, -rule[1]), rule[1]) + rule[1]
    count, D = rule[1], rule[2]
    half, E = count // 2, count // 4
    side, a = (half if x > 0 else 0), abs(x)
    if a < E:
        return side + a
    t = 0      # far bucket t begins where (a / E)^E >= (D / E)^t
    while t < half - E - 1 and a ** E * E ** (t + 1) >= D ** (t + 1) * E ** E:
        t += 1
    return side + E + t


def buckets(rule):
    return 2 * rule[1] + 1 if rule[0] == "exact" else rule[1]


def bucket_index(q_grid, k_grid, rows, cols, step=(1, 1), start=(0, 0)):
    """Table row of every pair, [n, m] int64."""
    out = torch.empty(q_grid[0] * q_grid[1], k_grid[0] * k_grid[1], dtype=torch.int64)
    memo_r, memo_c = {}, {}

    def look(memo, x, rule):
        if x not in memo:
            memo[x] = bucket_of(x, rule)
        return memo[x]

    kr = [(j // k_grid[1], j % k_grid[1]) for j in range(out.shape[1])]
    for i in range(out.shape[0]):
        r, c = i // q_grid[1] + start[0], i % q_grid[1] + start[1]
        out[i] = torch.tensor([look(memo_r, step[0] * a - r, rows) * buckets(cols) + look(memo_c, step[1] * b - c, cols)
                               for a, b in kr])
    return out


def attention(q, k, v, dout=None, *, scale, lens=None, table=None, index=None, dtype=torch.bfloat16):
    """Values and bounds.  q, dout [B, h, n, d], k, v [B, g, m, d], table
    [buckets, h] as the kernel got them; index [n, m] or a list of B of them.
    Returns {name: (value, bound)} for o, lse and, with dout, dq, dk, dv, dtable."""
    u, r = U[dtype], R[dtype]
    B, h, n, d = q.shape
    g, m = k.shape[1], k.shape[2]
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    tab = None if table is None else table.double().cpu()
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    o, Eo, lse, El = z(B, h, n, d), z(B, h, n, d), torch.full((B, h, n), -math.inf, dtype=torch.float64), z(B, h, n)
    if dout is not None:
        dout = dout.double().cpu()
        dq, Edq = z(B, h, n, d), z(B, h, n, d)
        dk, Edk, dv, Edv = (z(B, g, m, d) for _ in range(4))
        dt, Edt = (None, None) if tab is None else (torch.zeros_like(tab), torch.zeros_like(tab))
    for b in range(B):
        L = m if lens is None else max(0, min(int(lens[b]), m))
        if L == 0:
            continue
        for j in range(h):
            kk, vv, qq = k[b, j * g // h, :L], v[b, j * g // h, :L], q[b, j]
            s = scale * qq @ kk.T
            mag = scale * qq.abs() @ kk.abs().T
            if tab is not None:
                ix = (index[b] if isinstance(index, list) else index)[:, :L]
                s = s + tab[:, j][ix]
                mag = mag + tab[:, j][ix].abs().clamp(max=1e30)
            mag = torch.where(torch.isinf(s), 0.0, mag)
            l = torch.logsumexp(s, 1)
            some = l > -math.inf
            p = torch.where(some[:, None], torch.exp(s - torch.where(some, l, 0.0)[:, None]), 0.0)
            Es = u * (d + 8) * mag
            Esm = Es.amax(1)
            far = torch.where(p > 0, (s - torch.where(some, l, 0.0)[:, None]).abs(), 0.0)
            Ep = p * (Es + Esm[:, None] + u * (L + 8) + EX2 * 8 + 8 * u * far + 8 * 2.0 ** -24 * l.abs().clamp(max=1e30)[:, None]) + F
            o[b, j] = p @ vv
            Eo[b, j] = (Ep + (r + L * u) * p) @ vv.abs() + r * o[b, j].abs()
            lse[b, j] = l
            El[b, j] = Esm + u * (L + 8) + 8 * EX2 + 8 * 2.0 ** -24 * l.abs().clamp(max=1e30)
            if dout is None:
                continue
            do = dout[b, j]
            dp = do @ vv.T
            Edp = u * (d + 2) * (do.abs() @ vv.abs().T)
            delta = (p * dp).sum(1, keepdim=True)
            rounded = (do.abs() * Eo[b, j]).sum(1, keepdim=True) + u * (d + 2) * (do * o[b, j]).abs().sum(1, keepdim=True)
            summed = ((Ep + L * u * p) * dp.abs() + p * Edp).sum(1, keepdim=True)
            ds = p * (dp - delta)
            common = Ep * (dp - delta).abs() + p * (Edp + 4 * u * (dp.abs() + delta.abs())) + F
            Eds, Edx = common + p * torch.maximum(rounded, summed), common + p * summed
            dq[b, j] = scale * ds @ kk
            Edq[b, j] = scale * (Eds + (r + L * u) * ds.abs()) @ kk.abs() + r * dq[b, j].abs()
            at = j * g // h
            dk[b, at, :L] += scale * ds.T @ qq
            Edk[b, at, :L] += scale * (Eds + (r + n * u) * ds.abs()).T @ qq.abs()
            dv[b, at, :L] += p.T @ do
            Edv[b, at, :L] += (Ep + (r + n * u) * p).T @ do.abs()
            if tab is not None:
                dt[:, j].index_add_(0, ix.reshape(-1), ds.reshape(-1))
                Edt[:, j].index_add_(0, ix.reshape(-1), (Edx + 64 * u * p * (dp.abs() + delta.abs())).reshape(-1))
    tiny = 2.0 ** -126
    res = {"o": (o, 1.05 * Eo + tiny), "lse": (lse, 1.05 * El + tiny)}
    if dout is not None:
        res["dq"] = (dq, 1.05 * Edq + tiny)
        res["dk"] = (dk, 1.05 * (Edk + r * dk.abs()) + tiny)
        res["dv"] = (dv, 1.05 * (Edv + r * dv.abs()) + tiny)
        if tab is not None:
            res["dtable"] = (dt, 1.05 * Edt + tiny)
    return res


def assert_within(got, want, name):
    """got against (value, bound): finite or equal infinities, and inside the bound everywhere."""
    value, bound = want
    got = got.detach().double().cpu()
    assert got.shape == value.shape, name
    inf = torch.isinf(value)
    assert torch.equal(got[inf], value[inf]), "%s: infinities differ" % name
    off = torch.where(inf, 0.0, (got - value).abs() / bound)
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g times its bound" % (name, worst)   # NaN fails too
    return worst
