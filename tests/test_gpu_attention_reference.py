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


CASES = [
    # kernel, sequences' queries and keys, heads, heads of keys
    ("k_attn_few", [150, 7, 60], [150, 7, 60], 4, 2),
    ("k_attn_few", [1, 1, 1], [9000, 700, 60], 4, 2),          # in parts
    ("k_attn", [300] * 9 + [7, 203], [300] * 9 + [60, 203], 8, 8),
]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kernel, lens, klens, H, HK", CASES, ids=["rows", "parts", "tiles"])
@pytest.mark.parametrize("channels", [1, 2], ids=["lowest", "minus_inf"])
def test_first_keys_of_the_lowest_value(dt, kernel, lens, klens, H, HK, channels):
    """Keys padded with the type's lowest value, in one channel (scores of about that)
    or two (-inf): 40 at each sequence's start, all of a sequence where they are
    fewer, and 50 more further on.  They have no weight: out, lse and gradients are
    those of the other keys alone."""
    D = 64
    q, k, v, do = make(sum(lens), sum(klens), H, HK, D, dt, 2)
    q[..., :2] = 1.0
    k[..., :2] = 0.0
    keep = torch.ones(sum(klens), dtype=torch.bool)
    left, a = [], 0
    for m in klens:
        keep[a:a + (40 if m > 60 else m)] = False
        keep[a + 100:a + min(m, 150)] = False
        left.append(int(keep[a:a + m].sum()))
        a += m
    padded = (~keep).cuda()
    k[padded, :, :channels] = torch.finfo(dt).min
    o, ko = offs(lens), offs(klens)
    call = lambda: sp.spconv_attention(q, k, v, o, koffsets=ko, stats=True)
    assert_launches(call, f"{kernel}<{NAMES[dt]}, {D}>")
    out, lse = call()
    want = attention64(q, k[~padded], v[~padded], o, koffsets=offs(left), dout=do)
    # of scores of about -1e38 alone a sequence has a softmax, though none that says much
    some = torch.repeat_interleave(torch.tensor([n > 0 or channels == 2 for n in left]), torch.tensor(lens))
    beside = padded & torch.repeat_interleave(torch.tensor([n > 0 or channels == 2 for n in left]),
                                              torch.tensor(klens)).cuda()
    dq, dk, dv = sp.spconv_attention_grad(do, q, k, v, out, lse, o, koffsets=ko)
    for got, name in ((out, "out"), (lse, "lse"), (dq, "dq")):
        check(got.cpu()[some], [t[some] for t in want[name]], name)
    assert bool(torch.isfinite(out).all())
    for got, name in ((dk, "dk"), (dv, "dv")):
        check(got[~padded], want[name], name)
        assert bool((got[beside] == 0).all()), name


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kernel, lens, klens, H, HK", CASES, ids=["rows", "parts", "tiles"])
def test_infinite_first_keys(dt, kernel, lens, klens, H, HK):
    """Elements of -inf in the first 35 keys: scores of -inf, no weight."""
    D = 40
    q, k, v, _ = make(sum(lens), sum(klens), H, HK, D, dt, 3)
    q[..., 0] = q[..., 0].abs() + 0.5
    k[..., 0] = 0.0
    at = torch.cat([torch.arange(a, a + min(m, 35)) for a, m in
                    zip([sum(klens[:i]) for i in range(len(klens))], klens)])
    keep = torch.ones(sum(klens), dtype=torch.bool)
    keep[at] = False
    k[at.cuda(), :, 0] = -math.inf
    o = offs(lens)
    call = lambda: sp.spconv_attention(q, k, v, o, koffsets=offs(klens), stats=True)
    assert_launches(call, f"{kernel}<{NAMES[dt]}, 64>")
    out, lse = call()
    want = attention64(q, k[keep.cuda()], v[keep.cuda()], o, koffsets=offs([max(0, m - 35) for m in klens]))
    check(out, want["out"], "out")
    check(lse, want["lse"], "lse")
