"""Attention's bf16 gradients where no sequence has more than 256 keys.

There p and ds are operands in two bf16 parts, hi = bf16(x) and lo = bf16(x - hi),
which leave 2^-8 2^-8 = 2^-16 of x, and delta is a sum over the keys in 32 bits, not
dout times the rounded output.  So a gradient is off by its own rounding, h = 2^-8 of
itself, and by terms that are small beside it.  With u = 2^-24, e the relative error
of a weight (attn_ref; the statistics' errors included), m keys, n queries:

  dp     (D + 2) u sum |dout v|
  delta  sum_j p (e |dp| + the error of dp) + (m + 4) u sum_j p |dp|
  ds     e |ds| + p (the errors of dp and delta + 2 u (|dp| + |delta|))
  dq     scale sum_j ((2^-16 + (m + 4) u) |ds| + its error) |k|, dk the same over the
         queries (n G of them), dv with p in place of ds and |dout| of |k|

each with half a step of the result beside it.
"""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu
U, H, TWO = 2.0 ** -24, 2.0 ** -8, 2.0 ** -16
BF = torch.bfloat16


def gradient64(q, k, v, dout, lens, causal):
    """{name: (value, bound)} over sequences of equal queries and keys, one after the other."""
    q, k, v, dout = (t.double().cpu() for t in (q, k, v, dout))
    D, G = q.shape[2], q.shape[1] // k.shape[1]
    scale = D ** -0.5
    r = {n: (torch.zeros_like(t), torch.zeros_like(t)) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    a = 0
    for n in lens:
        hidden = torch.ones(n, n).triu(1).bool() if causal else torch.zeros(n, n).bool()
        for g in range(q.shape[1]):
            Q, K, V, O = q[a:a + n, g], k[a:a + n, g // G], v[a:a + n, g // G], dout[a:a + n, g]
            s = (Q @ K.T * scale).masked_fill(hidden, -torch.inf)
            l = torch.logsumexp(s, 1, keepdim=True)
            p = torch.exp(s - l)
            e = 2 * ((D + 2) * U * scale * (Q.abs() @ K.abs().T).masked_fill(hidden, 0)).amax(1, keepdim=True)
            e = e + 8 * U * (1 + s.masked_fill(hidden, 0).abs().amax(1, keepdim=True) + l.abs())
            e = 2 * e + (n + 4) * U + 6 * U * l.abs()
            dp, dpe = O @ V.T, (D + 2) * U * (O.abs() @ V.abs().T)
            delta = (p * dp).sum(1, keepdim=True)
            deltae = (p * (e * dp.abs() + dpe) + (n + 4) * U * p * dp.abs()).sum(1, keepdim=True)
            ds = p * (dp - delta)
            dse = e * ds.abs() + p * (dpe + deltae + 2 * U * (dp.abs() + delta.abs()))
            left = lambda m, x, xe: (TWO + (m + 4) * U) * x.abs() + xe
            for name, row, d, err in (
                    ("dq", g, ds @ K, left(n, ds, dse) @ K.abs()),
                    ("dk", g // G, ds.T @ Q, left(n * G, ds, dse).T @ Q.abs()),
                    ("dv", g // G, p.T @ O / scale, left(n * G, p, e * p).T @ O.abs() / scale)):
                r[name][0][a:a + n, row] += scale * d
                r[name][1][a:a + n, row] += scale * err
        a += n
    return {n: (d, e + H * d.abs() + 1e-37) for n, (d, e) in r.items()}


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[2], [2] * 40, [1, 3, 31, 32, 33], [200, 17], [256] * 5], ids=lambda v: f"{len(v)}x{v[0]}")
def test_short_sequences(lens, causal, D):
    print(lens[:5], causal, D, flush=True)
    g = torch.Generator().manual_seed(sum(lens) + D)
    N = sum(lens)
    q, dout = (torch.randn(N, 4, D, generator=g).to(BF).cuda() for _ in range(2))
    k, v = (torch.randn(N, 2, D, generator=g).to(BF).cuda() for _ in range(2))
    o = torch.tensor([0] + lens).cumsum(0).int().cuda()
    out, lse = sp.spconv_attention(q, k, v, o, causal=causal, stats=True)
    got = sp.spconv_attention_grad(dout, q, k, v, out, lse, o, causal=causal)
    torch.cuda.synchronize()
    want = gradient64(q, k, v, dout, lens, causal)
    for name, t in zip(("dq", "dk", "dv"), got):
        d, bound = want[name]
        off = (t.double().cpu() - d).abs() / bound
        assert float(off.max()) <= 1, f"{name}: {float(off.max()):.3g} of the bound"
