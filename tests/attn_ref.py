"""Attention and its gradient in 64 bits on the host, with bounds on what the
kernels' arithmetic may be off by.

u is half a step of 32 bits (2^-24), h half a step of the element type: what is
rounded to it once is off by h of itself.

Scores: sums of D products in 32 bits, times scale: off by ds <= (D + 2) u scale
sum |q k|.  A weight exp(s - lse) is off by ds, the rounding of its exponent
(terms as large as |s| and |lse|) and of the exponential, a few u: relatively
  e = 2 ds + 8 u (1 + |s| + |lse|), over the whole row.
out: weights rounded by h, the sum over L keys in 32 bits, one rounding:
  |out| h + (e + h + (L + 4) u) sum_j p |v|
dv:  |dv| h + (e + h + (n + 4) u) sum_i p |dout|      (n queries)
ds = p (dp - delta): dp is off by (D + 2) u sum |dout v|, delta by as much and by
  the error of the output that it is made from:
  e p |dp - delta| + p ((D + 4) u (sum |dout v| + sum |dout out|) + sum |dout| d_out) + h |ds|
dq, dk: scale sums of it with |k|, |q|, the sum's own rounding, one rounding.
"""
import math

import torch

U = 2.0 ** -24
H = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def lens_of(offsets):
    o = offsets.tolist()
    return list(zip(o[:-1], o[1:]))


def attention64(q, k, v, offsets, koffsets=None, order=None, korder=None, causal=False, scale=None, dout=None,
                given=None):
    """Returns {name: (value, bound)} for out, lse and, with dout, dq, dk, dv;
    rows outside the sequences hold NaN.  given: the kernel's (out, lse), whose own
    errors are then what the gradient's inputs are off by."""
    h = H[q.dtype]
    q, k, v = (t.detach().double().cpu() for t in (q, k, v))
    N, Hq, D = q.shape
    M, HK = k.shape[:2]
    scale = D ** -0.5 if scale is None else scale
    if koffsets is None:
        koffsets, korder = offsets, order
    qi = order.long().cpu() if order is not None else torch.arange(N)
    ki = korder.long().cpu() if korder is not None else torch.arange(M)
    nan = float("nan")
    out, oe = torch.full_like(q, nan), torch.full_like(q, nan)
    lse, le = torch.full((N, Hq), nan, dtype=torch.float64), torch.full((N, Hq), nan, dtype=torch.float64)
    if dout is not None:
        dout = dout.detach().double().cpu()
        dq, dqe = torch.full_like(q, nan), torch.full_like(q, nan)
        dk, dke, dv, dve = (torch.full_like(k, nan) for _ in range(4))
    for (a, b), (c, d) in zip(lens_of(offsets.cpu()), lens_of(koffsets.cpu())):
        rq, rk = qi[a:b], ki[c:d]
        n, m = b - a, d - c
        if dout is not None:
            for t in (dk, dke, dv, dve):
                t[rk] = 0.0
        hidden = torch.zeros(n, m, dtype=torch.bool)
        if causal:
            hidden = torch.arange(m)[None, :] > torch.arange(n)[:, None] + (m - n)
        for g in range(Hq):
            kh, vh, qh = k[rk, g // (Hq // HK)], v[rk, g // (Hq // HK)], q[rq, g]
            out[rq, g], oe[rq, g], lse[rq, g], le[rq, g] = 0.0, 0.0, -math.inf, 0.0
            if dout is not None:
                dq[rq, g], dqe[rq, g] = 0.0, 0.0
            if n == 0 or m == 0:
                continue
            s = (qh @ kh.T * scale).masked_fill(hidden, -math.inf)
            l = torch.logsumexp(s, 1)
            blind = l == -math.inf
            l0 = l.masked_fill(blind, 0.0)
            p = torch.exp(s - l0[:, None])
            sa = s.masked_fill(hidden, 0.0).abs()
            serr = (D + 2) * U * scale * (qh.abs() @ kh.abs().T).masked_fill(hidden, 0.0)
            e = 2 * serr.amax(1) + 8 * U * (1 + sa.amax(1) + l0.abs())
            o = p @ vh
            pv = p @ vh.abs()
            out[rq, g], lse[rq, g] = o, l
            oe[rq, g] = o.abs() * h + (e[:, None] + h * (h > U) + (m + 4) * U) * pv
            le[rq, g] = e + (m + 4) * U
            if dout is None:
                continue
            do = dout[rq, g]
            dp, delta = do @ vh.T, (do * o).sum(1, keepdim=True)
            ds = p * (dp - delta)
            derr = (D + 4) * U * (do.abs() @ vh.abs().T + (do * o).abs().sum(1, keepdim=True)) \
                + (do.abs() * oe[rq, g]).sum(1, keepdim=True)
            e2 = e[:, None] + le[rq, g][:, None] + l0.abs()[:, None] * 4 * U
            dse = e2 * ds.abs() + p * derr + h * (h > U) * (ds.abs() + p * derr)
            dq[rq, g] = scale * ds @ kh
            dqe[rq, g] = scale * (dse + (m + 4) * U * ds.abs()) @ kh.abs()
            dk[rk, g // (Hq // HK)] += scale * ds.T @ qh
            dke[rk, g // (Hq // HK)] += scale * (dse + (n * Hq // HK + 4) * U * ds.abs()).T @ qh.abs()
            dv[rk, g // (Hq // HK)] += p.T @ do
            dve[rk, g // (Hq // HK)] += ((e2 + h * (h > U) + (n * Hq // HK + 4) * U) * p).T @ do.abs()
    r = {"out": (out, oe), "lse": (lse, le + 2 * U * lse.abs().nan_to_num(posinf=0.0))}
    if dout is not None:
        for name, t, err in (("dq", dq, dqe), ("dk", dk, dke), ("dv", dv, dve)):
            r[name] = (t, err + h * t.abs())
    return r


def check(got, want, what, untouched=None):
    """got within the bound of want; rows that want holds NaN in are `untouched`."""
    value, bound = want
    got = got.double().cpu()
    inside = ~torch.isnan(value)
    if untouched is not None:
        assert bool((got[~inside] == untouched).all()), f"{what}: rows behind the sequences were written"
    value, bound, got = value[inside], bound[inside], got[inside]
    same = value == got
    bad = ~same & ~((got - value).abs() <= bound * 1.0 + 1e-37)
    if bool(bad.any()):
        i = bad.nonzero()[0]
        worst = ((got - value).abs() / (bound + 1e-300))[bad].max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, the worst by {float(worst):.3g} of "
                             f"the bound, first {got[i].item()} for {value[i].item()}")
