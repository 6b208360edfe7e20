"""The reference that a query's exponentials are taken against, in both forward
kernels (16 and 128 rows a workgroup): it is the maximum of the first keys, and
is taken again where those do not do.

Whether a query's is taken again goes by the keys that it sees.  A key hidden
from it, however large, must not change its bits, although other queries of its
tile see the key.
"""
import math

import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp
from attn_ref import attention64, check
from kernel_names import assert_launches

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = {BF: "bf16", F32: "f32"}


def offs(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def make(N, M, H, HK, D, dt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()
    return r(N, H, D), r(M, HK, D), r(M, HK, D), r(N, H, D)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kernel, seqs, heads", [("k_attn_few", 3, 2), ("k_attn", 10, 8)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e30, -3e38])
def test_hidden_keys_leave_the_reference(dt, kernel, seqs, heads, value):
    """Sequences of 300 rows, causal, keys from row 200 on that overflow the weights of
    the queries that see them: the 200 before keep their bits."""
    L, cut, D = 300, 200, 64
    q, k, v, _ = make(seqs * L, seqs * L, heads, heads, D, dt, 1)
    o = offs([L] * seqs)
    call = lambda k, v: sp.spconv_attention(q, k, v, o, causal=True, stats=True)
    assert_launches(lambda: call(k, v), f"{kernel}<{NAMES[dt]}, {D}>")
    want, lse = call(k, v)
    for keys, values in ((True, False), (False, True), (True, True)):
        k2, v2 = k.clone(), v.clone()
        for t, use in ((k2, keys), (v2, values)):
            if use:
                t.view(seqs, L, heads, D)[:, cut::3] = value
        got, lse2 = call(k2, v2)
        first = lambda t: t.view(seqs, L, *t.shape[1:])[:, :cut]
        assert torch.equal(first(got), first(want)) and torch.equal(first(lse2), first(lse)), (keys, values)
