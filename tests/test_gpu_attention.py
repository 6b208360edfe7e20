"""Attention within packed sequences against 64 bits: types, widths, grouped
heads, lengths from none to long ones, orders, strides, empty rows; bounds as
derived in attn_ref."""
import math

import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp
from attn_ref import attention64, check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def offs(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def make(N, M, H, HK, D, dt, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed * 1000003 + N * 31 + M)
    r = lambda *s: torch.randn(*s, generator=g)
    return [t.to(dt).cuda() for t in (r(N, H, D) * spread, r(M, HK, D), r(M, HK, D), r(N, H, D))] + [g]


def both(q, k, v, dout, offsets, **kw):
    """Forward and gradient against 64 bits; untouched rows stay."""
    print("forward", tuple(q.shape), tuple(k.shape), q.dtype, {a: b for a, b in kw.items() if not torch.is_tensor(b)},
          flush=True)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=q.device)
    o, lse = sp.spconv_attention(q, k, v, offsets, stats=True, out=out, **kw)
    torch.cuda.synchronize()
    want = attention64(q, k, v, offsets, dout=dout, **kw)
    check(o, want["out"], "out", untouched=7.0)
    check(lse, want["lse"], "lse")
    grads = [torch.full(t.shape, 7.0, dtype=t.dtype, device=t.device) for t in (q, k, v)]
    print("gradient", flush=True)
    grads = sp.spconv_attention_grad(dout, q, k, v, o, lse, offsets, grads=grads, **kw)
    torch.cuda.synchronize()
    for name, t in zip(("dq", "dk", "dv"), grads):
        check(t, want[name], name, untouched=7.0)
    return o, lse, grads


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 32, 40, 64, 96, 104, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_widths(dt, D, causal):
    q, k, v, do, _ = make(203, 203, 4, 2, D, dt, seed=D)
    both(q, k, v, do, offs([70, 0, 1, 132]), causal=causal)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H, HK", [(1, 1), (3, 1), (6, 2), (8, 8), (32, 2), (40, 1)])
def test_groups_of_heads(dt, H, HK):
    q, k, v, do, _ = make(77, 77, H, HK, 32, dt, seed=H)
    both(q, k, v, do, offs([40, 37]), causal=True)


@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [0, 5, 0], [31, 32, 33], [63, 64, 65], [127, 128, 129], [511, 0, 2],
                                  [1] * 150, [700]], ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(lens, causal):
    N = sum(lens)
    q, k, v, do, _ = make(N, N, 2, 1, 64, BF, seed=len(lens))
    both(q, k, v, do, offs(lens), causal=causal)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens, klens", [([1, 1, 1], [5, 700, 0]), ([1], [2049]), ([3, 0, 40, 9], [0, 17, 200, 4]),
                                         ([200, 1], [3, 64]), ([2500], [7])], ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_keys_of_their_own(dt, lens, klens, causal):
    """Queries without keys, keys without queries, causal rows that see nothing."""
    q, k, v, do, _ = make(sum(lens), sum(klens), 4, 2, 64, dt, seed=7)
    o, lse, _ = both(q, k, v, do, offs(lens), koffsets=offs(klens), causal=causal)
    a = 0
    for n, m in zip(lens, klens):
        blind = n if m == 0 else max(0, n - m) if causal else 0
        assert bool((o[a:a + blind] == 0).all()) and bool((lse[a:a + blind] == -math.inf).all())
        assert bool(torch.isfinite(lse[a + blind:a + n]).all())
        a += n


@pytest.mark.parametrize("dt, D, G", [(BF, 128, 4), (BF, 32, 1), (F32, 64, 2)])
def test_single_queries_and_long_keys(dt, D, G):
    """Keys split over workgroups: few queries, 20,001 and 3 keys."""
    q, k, v, do, _ = make(2, 20004, 2 * G, 2, D, dt, seed=3)
    assert sp.spconv_attention_workspace_size(2, 20004, 2, 2 * G, 2, D, dt == BF) > 0
    both(q, k, v, do, offs([1, 1]), koffsets=offs([20001, 3]), causal=True)


def test_many_queries_and_few_keys():
    """The keys' gradient splits the queries."""
    q, k, v, do, _ = make(9000, 20, 2, 1, 32, BF, seed=4)
    both(q, k, v, do, offs([8900, 100]), koffsets=offs([13, 7]))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_order_and_rows_behind(dt):
    N = 300
    q, k, v, do, g = make(N, N, 4, 2, 32, dt, seed=9)
    order = torch.randperm(N, generator=g).to(torch.int32).cuda()
    both(q, k, v, do, offs([100, 0, 150]), order=order, causal=True)      # 50 rows in no sequence
    M = 400
    _, k, v, _, _ = make(N, M, 4, 2, 32, dt, seed=10)
    korder = torch.randperm(M, generator=g).to(torch.int32).cuda()
    both(q, k, v, do, offs([100, 0, 150]), koffsets=offs([30, 20, 260]), order=order, korder=korder)


def test_strided_heads():
    """Queries, keys and values as parts of one projection; gradients into the
    parts of its gradient."""
    N, H, D = 150, 3, 40
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(N, 3, H, D, generator=g).to(BF).cuda()
    do = torch.randn(N, H, D, generator=g).to(BF).cuda()
    q, k, v = qkv.unbind(1)
    o = offs([100, 50])
    a, lse = sp.spconv_attention(q, k, v, o, causal=True, stats=True)
    b, lse2 = sp.spconv_attention(q.contiguous(), k.contiguous(), v.contiguous(), o, causal=True, stats=True)
    assert torch.equal(a, b) and torch.equal(lse, lse2)
    dqkv = torch.zeros_like(qkv)
    sp.spconv_attention_grad(do, q, k, v, a, lse, o, causal=True, grads=dqkv.unbind(1))
    want = sp.spconv_attention_grad(do, q.contiguous(), k.contiguous(), v.contiguous(), a, lse, o, causal=True)
    for x, y in zip(dqkv.unbind(1), want):
        assert torch.equal(x, y)
    # heads before rows, and a broadcast key
    t = qkv[:, 0].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(sp.spconv_attention(t, k, v, o), sp.spconv_attention(q, k, v, o))
    ke = k[:1].expand(N, H, D)
    assert torch.equal(sp.spconv_attention(q, ke, v, o), sp.spconv_attention(q, ke.contiguous(), v, o))
    # odd strides are copied
    odd = torch.randn(N, H, D + 1, device="cuda").to(BF)[..., :D]
    assert torch.equal(sp.spconv_attention(odd, k, v, o), sp.spconv_attention(odd.contiguous(), k, v, o))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3e38])
def test_hidden_rows_have_no_effect(dt, value):
    """What a query does not see may hold anything, in the same tile or not, and
    behind the sequence; likewise the gradients of a query that a key is hidden
    from."""
    N, cut = 200, 101
    q, k, v, do, _ = make(N, N, 2, 1, 64, dt, seed=11)
    o = offs([150])
    clean, lse = sp.spconv_attention(q, k, v, o, causal=True, stats=True)
    k2, v2, q2, do2 = k.clone(), v.clone(), q.clone(), do.clone()
    for t in (k2, v2):
        t[cut::7] = value
    got, lse2 = sp.spconv_attention(q, k2, v2, o, causal=True, stats=True)
    assert torch.equal(got[:cut], clean[:cut]) and torch.equal(lse2[:cut], lse[:cut])
    want = sp.spconv_attention_grad(do, q, k, v, clean, lse, o, causal=True)
    got = sp.spconv_attention_grad(do, q, k2, v2, clean, lse, o, causal=True)
    assert torch.equal(got[0][:cut], want[0][:cut])
    # queries before a key do not see it
    for t in (q2, do2):
        t[:cut:7] = value
    got = sp.spconv_attention_grad(do2, q2, k, v, clean, lse, o, causal=True)
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[cut:150], b[cut:150])


def test_infinite_values_reach_those_that_see_them():
    q, k, v, do, _ = make(40, 40, 1, 1, 32, F32, seed=12)
    v[20, 0, 3] = float("inf")
    out = sp.spconv_attention(q, k, v, offs([40]), causal=True)
    assert bool(torch.isfinite(out[:20]).all())
    assert bool((out[20:, 0, 3] == float("inf")).all())
    assert int((~torch.isfinite(out)).sum()) == 20
    q[5] = float("nan")
    out, lse = sp.spconv_attention(q, k, v, offs([40]), causal=True, stats=True)
    assert bool(torch.isnan(out[5]).all()) and bool(torch.isnan(lse[5]).all())
    assert bool(torch.isfinite(out[6:20]).all()) and bool(torch.isfinite(lse[6:]).all())


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_large_and_growing_scores(dt):
    """Scores of thousands, ever larger along the keys: the running reference
    follows."""
    q, k, v, do, _ = make(130, 130, 1, 1, 32, dt, seed=13)
    k = k * torch.linspace(1, 60, 130, device="cuda")[:, None, None].to(dt)
    want = attention64(q, k, v, offs([130]), scale=2.0)
    out, lse = sp.spconv_attention(q, k, v, offs([130]), scale=2.0, stats=True)
    check(out, want["out"], "out")
    check(lse, want["lse"], "lse")


def test_single_keys_give_zero_gradients():
    """A softmax over one key is 1 whatever the score: dq and dk are 0."""
    for dt in (BF, F32):
        q, k, v, do, _ = make(90, 90, 4, 2, 48, dt, seed=14)
        o = offs([1] * 90)
        out, lse = sp.spconv_attention(q, k, v, o, stats=True)
        assert torch.equal(out, v.repeat_interleave(2, 1))
        dq, dk, dv = sp.spconv_attention_grad(do, q, k, v, out, lse, o)
        assert bool((dq == 0).all()) and bool((dk == 0).all())


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(5)
    N, H, HK, D = 60, 2, 1, 16
    q, k, v, do = (torch.randn(*s, generator=g).cuda() for s in ((N, H, D), (N, HK, D), (N, HK, D), (N, H, D)))
    o = offs([25, 35])
    out, lse = sp.spconv_attention(q, k, v, o, causal=True, stats=True)
    grads = sp.spconv_attention_grad(do, q, k, v, out, lse, o, causal=True)
    f = lambda *t: float((sp.spconv_attention(*t, o, causal=True).double() * do.double()).sum())
    for i, t in enumerate((q, k, v)):
        d = torch.randn(t.shape, generator=g).cuda()
        step = 1e-2
        args = [q, k, v]
        args[i] = t + step * d
        hi = f(*args)
        args[i] = t - step * d
        lo = f(*args)
        want = float((grads[i].double() * d.double()).sum())
        # third-order term step^2 / 6 f''' and 32-bit outputs over 2 step
        size = float(do.double().norm()) * float(d.double().norm())
        assert abs((hi - lo) / (2 * step) - want) <= size * (step ** 2 + 2 ** -24 * 8 / step), i


def test_same_bits_twice_and_empty():
    q, k, v, do, _ = make(1000, 1000, 4, 2, 64, BF, seed=15)
    o = offs([600, 400])
    a = both(q, k, v, do, o, causal=True)
    b = both(q, k, v, do, o, causal=True)
    for x, y in zip((a[0], a[1], *a[2]), (b[0], b[1], *b[2])):
        assert torch.equal(x, y)
    e = torch.zeros(0, 4, 64, dtype=BF, device="cuda")
    ke = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    z = offs([0, 0])
    out, lse = sp.spconv_attention(e, ke, ke, z, stats=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    dq, dk, dv = sp.spconv_attention_grad(e, e, k, v, e, lse, z, koffsets=o)
    assert bool((dk == 0).all()) and bool((dv == 0).all())
    out, lse = sp.spconv_attention(q, ke, ke, o, koffsets=z, stats=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    dq, dk, dv = sp.spconv_attention_grad(do, q, ke, ke, out, lse, o, koffsets=z)
    assert bool((dq == 0).all()) and dk.shape == (0, 2, 64)
