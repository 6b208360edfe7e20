"""bf16 attention of few rows (16 a workgroup), forward: the weights are operands
in two bf16 parts, hi = bf16(w) and lo = bf16(w - hi), which leave 2^-8 2^-8 = 2^-16
of w, so that an output is off by its own rounding, h = 2^-8 of itself, and by terms
that are small beside it.  With u = 2^-24, m keys and e the relative error of a
weight (scores off by (D + 2) u scale sum |q k|, exponents and exponentials by a few
u; attn_ref):

  |out| h + (e + 2^-16 + (m + 4) u) sum_j p |v|
"""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp
from kernel_names import assert_launches

pytestmark = pytest.mark.gpu
U, H, TWO = 2.0 ** -24, 2.0 ** -8, 2.0 ** -16
BF = torch.bfloat16


def offs(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


@pytest.mark.parametrize("D", [24, 32, 64, 96, 128])
@pytest.mark.parametrize("lens, klens, causal", [([70, 0, 1, 132, 300], [70, 0, 1, 132, 300], True),
                                                 ([17, 200], [33, 1500], False),
                                                 ([1, 1, 1], [9000, 31, 700], False)], ids=["rows", "keys", "parts"])
def test_weights_in_two_parts(D, lens, klens, causal):
    N, M, heads, HK = sum(lens), sum(klens), 4, 2
    g = torch.Generator().manual_seed(N + M + D)
    q, k, v = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((N, heads, D), (M, HK, D), (M, HK, D)))
    call = lambda: sp.spconv_attention(q, k, v, offs(lens), koffsets=offs(klens), causal=causal)
    assert_launches(call, f"k_attn_few<bf16, {(D + 31) // 32 * 32}>")
    out = call().double().cpu()
    q, k, v = (t.double().cpu() for t in (q, k, v))
    scale, a, b = D ** -0.5, 0, 0
    for n, m in zip(lens, klens):
        hidden = torch.ones(n, m).triu(m - n + 1).bool() if causal else torch.zeros(n, m).bool()
        for h in range(heads if n * m else 0):
            Q, K, V = q[a:a + n, h], k[b:b + m, h // 2], v[b:b + m, h // 2]
            s = (Q @ K.T * scale).masked_fill(hidden, -torch.inf)
            l = torch.logsumexp(s, 1, keepdim=True)
            p = torch.exp(s - l)
            e = 2 * (D + 2) * U * (scale * (Q.abs() @ K.abs().T)).masked_fill(hidden, 0).amax(1, keepdim=True)
            e = e + 8 * U * (1 + s.masked_fill(hidden, 0).abs().amax(1, keepdim=True) + l.abs())
            want = p @ V
            bound = H * want.abs() + (e + TWO + (m + 4) * U) * (p @ V.abs())
            off = float(((out[a:a + n, h] - want).abs() / bound).max())
            assert off <= 1, f"{n} rows, {m} keys, head {h}: {off:.3g} of the bound"
        a, b = a + n, b + m
