"""Attention over tensors past 2 GiB: keys in their rows' order and through a list
of rows, and rows far apart.  The reference is the definition in 64 bits on the
GPU, in pieces; the bound is that of attn_ref with its sums over the keys taken
as they are: bf16 weights and outputs rounded once (2^-8 each), scores off by
(D + 2) 2^-24 of their absolute sum.
"""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp
from attn_ref import attention64, check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def definition(q, k, v, rows):
    """out, sum p |v| and the largest score bound for one query, keys k[rows]."""
    D = q.shape[-1]
    HK, G = k.shape[1], q.shape[0] // k.shape[1]
    qd = q.double().view(HK, G, D)
    s, bound = [], 0.0
    for r in rows.split(1 << 20):
        kk = k[r].double()
        s.append(torch.stack([qd[h] @ kk[:, h].T for h in range(HK)]) * D ** -0.5)
        bound = max(bound, float((q.double().abs().max() * kk.abs().sum(2).max()) * D ** -0.5))
    p = torch.softmax(torch.cat(s, 2), 2)
    out, pv, at = torch.zeros_like(qd), torch.zeros_like(qd), 0
    for r in rows.split(1 << 20):
        vv = v[r].double()
        for h in range(HK):
            out[h] += p[h, :, at:at + len(r)] @ vv[:, h]
            pv[h] += p[h, :, at:at + len(r)] @ vv[:, h].abs()
        at += len(r)
    return out.view(-1, D), pv.view(-1, D), 2 * (D + 2) * 2.0 ** -24 * bound


@pytest.mark.parametrize("listed", [False, True])
def test_long_cache(listed):
    M, HK, H, D = 9_000_000, 2, 4, 64            # 2.3 GB of keys, as much of values
    assert M * HK * D * 2 > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(M, HK, D, generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(2, H, D, generator=g, device="cuda").to(BF)
    # one short sequence at the end, one long before it
    cut = M - 1000
    off = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    ko = torch.tensor([0, cut, M], dtype=torch.int32, device="cuda")
    order = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda") if listed else None
    print("forward", listed, flush=True)
    out = sp.spconv_attention(q, k, v, off, koffsets=ko, korder=order, causal=True)
    torch.cuda.synchronize()
    at = torch.arange(M, device="cuda") if order is None else order.long()
    for i, rows in enumerate((at[:cut], at[cut:])):
        want, pv, e = definition(q[i], k, v, rows)
        bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + e + len(rows) * 2.0 ** -24) * pv
        assert bool(((out[i].double() - want).abs() <= bound).all()), i


def test_rows_far_apart_are_copied():
    """Rows more than 16 MiB apart: the binding copies them, the library refuses."""
    big = torch.zeros(3, (1 << 23) + 64, device="cuda", dtype=BF)
    far = big[:, :64].view(3, 1, 64)
    far.copy_(torch.randn(3, 1, 64, device="cuda"))
    assert far.stride(0) * 2 > 1 << 24
    o = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    assert torch.equal(sp.spconv_attention(far, far, far, o), sp.spconv_attention(*[far.contiguous()] * 3, o))
    with pytest.raises(ValueError):
        sp.spconv_attention(far, far, far, o, out=far)


def test_heads_far_apart():
    """Heads of whole tensors one after the other: past 2 GiB from first to last.

    The same rows in a small tensor need not give the same bits: which kernel a call
    takes goes by its rows in all per sequence (2,200,000 here, 300 there), since the
    offsets are on the device, and the kernels add in different orders.  Both are
    within attn_ref's bound of the definition."""
    N, H, D = 2_200_000, 8, 64
    t = torch.zeros(H, N, D, dtype=BF, device="cuda")
    assert t.numel() * 2 > 1 << 31
    n = 300
    g = torch.Generator(device="cuda").manual_seed(2)
    for i in range(H):
        t[i, :n] = torch.randn(n, D, generator=g, device="cuda")
    q = t.transpose(0, 1)
    o = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    k = torch.zeros(N, 1, D, dtype=BF, device="cuda")
    k[:n] = torch.randn(n, 1, D, generator=g, device="cuda")
    small = [x[:n].contiguous() for x in (q, k)]
    for qq, kk in ((q, k), small):
        out, lse = sp.spconv_attention(qq, kk, kk, o, causal=True, stats=True)
        grads = sp.spconv_attention_grad(qq, qq, kk, kk, out, lse, o, causal=True)
        want = attention64(*[small[i] for i in (0, 1, 1)], o, causal=True, dout=small[0])
        for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            check(got[:n], want[name], f"{name} of {len(qq)} rows")
