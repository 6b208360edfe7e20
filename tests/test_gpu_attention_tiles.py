"""The attention kernels that large calls take (128 rows a workgroup that shares
tiles of the other axis: k_attn, k_attn_dq<.., 0>, k_attn_dkv<.., 0>) against 64
bits: types, widths, masks, lists of rows, keys of their own, long and empty
sequences, hidden and infinite keys.  Each test says which kernels it is meant
for; bounds as derived in attn_ref."""
import math

import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp
from attn_ref import attention64, check
from kernel_names import assert_launches

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = {BF: "bf16", F32: "f32"}
# empty and single rows, ends around tiles of 32, 64 and 128 rows and 256 keys
LENS = [300, 40, 0, 513, 1, 129, 290, 64, 257, 33, 406, 128, 77, 65, 31, 0, 256, 220]
KLENS = [1, 300, 70, 129, 0, 513, 33, 64, 290, 257, 128, 406, 200, 3, 31, 9, 600, 0]


def offs(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def make(N, M, H, HK, D, dt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    q, k, v, do = (t.to(dt).cuda() for t in (r(N, H, D) * 1.5, r(M, HK, D), r(M, HK, D), r(N, H, D)))
    perm = lambda n: torch.randperm(n, generator=g).to(torch.int32).cuda()
    return q, k, v, do, perm


def width(D):
    return (D + 31) // 32 * 32


def both(q, k, v, do, offsets, split=False, **kw):
    """Forward and gradient, from the kernels that share tiles, against 64 bits; rows
    behind the sequences stay."""
    dt, D = q.dtype, q.shape[2]
    what = f"<{NAMES[dt]}, {width(D)}"
    out = torch.full(q.shape, 7.0, dtype=dt, device="cuda")
    grads = [torch.full(t.shape, 7.0, dtype=dt, device="cuda") for t in (q, k, v)]
    print("forward", tuple(q.shape), tuple(k.shape), dt, sorted(kw), flush=True)
    o, lse = sp.spconv_attention(q, k, v, offsets, stats=True, out=out, **kw)
    torch.cuda.synchronize()
    print("gradient", flush=True)
    sp.spconv_attention_grad(do, q, k, v, o, lse, offsets, grads=grads, **kw)
    torch.cuda.synchronize()
    if not split:
        assert_launches(lambda: sp.spconv_attention(q, k, v, offsets, out=out, **kw), f"k_attn{what}>")
    assert_launches(lambda: sp.spconv_attention_grad(do, q, k, v, o, lse, offsets, grads=grads, **kw),
                    f"k_attn_dq{what}, 0>", f"k_attn_dkv{what}, 0>", *[f"k_attn_sum<{NAMES[dt]}>"] * split)
    want = attention64(q, k, v, offsets, dout=do, **kw)
    check(o, want["out"], "out", untouched=7.0)
    check(lse, want["lse"], "lse")
    for name, t in zip(("dq", "dk", "dv"), grads):
        check(t, want[name], name, untouched=7.0)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 32, 40, 64, 96, 104, 128])
@pytest.mark.parametrize("form", ["full", "causal", "causal_order", "keys", "causal_keys_order"])
def test_every_form(dt, D, form):
    N = sum(LENS) + 25                       # 25 rows in no sequence
    M = sum(KLENS) + 15 if "keys" in form else N
    q, k, v, do, perm = make(N, M, 8, 8, D, dt, D + len(form))
    kw = {"causal": "causal" in form}
    if "order" in form:
        kw["order"] = perm(N)
    if "keys" in form:
        kw["koffsets"] = offs(KLENS)
        if "order" in form:
            kw["korder"] = perm(M)
    both(q, k, v, do, offs(LENS), **kw)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H, HK", [(8, 2), (12, 4), (40, 8), (32, 1)])
@pytest.mark.parametrize("order", [False, True])
def test_groups_of_heads(dt, H, HK, order):
    """Tiles of queries that are whole positions, and not (groups of 3 and 5)."""
    lens = LENS + [300] * (4 if HK < 8 else 0) + [60] * (15 if HK == 1 else 0)
    N = sum(lens)
    q, k, v, do, perm = make(N, N, H, HK, 32, dt, H)
    both(q, k, v, do, offs(lens), causal=True, order=perm(N) if order else None)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_long_axis_in_parts(dt, D):
    """Few long sequences: the gradients' other axis is split over workgroups."""
    lens = [700, 1300, 0, 650]
    q, k, v, do, perm = make(sum(lens), sum(lens), 8, 4, D, dt, D)
    both(q, k, v, do, offs(lens), split=True, causal=True, order=perm(sum(lens)))
    both(q, k, v, do, offs(lens), split=True)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_listed_rows_of_large_tensors(dt):
    """Rows 1 MiB apart, tensors past 2 GiB: listed rows are read at 64-bit addresses."""
    N, H, D = sum(LENS), 8, 64
    q, k, v, do, perm = make(N, N, H, H, D, dt, 5)
    step = (1 << 20) // q.element_size()
    far = []
    for t in (q, k, v):
        big = torch.empty(N, step, dtype=dt, device="cuda")
        assert big.numel() * big.element_size() > 1 << 31
        far.append(big[:, :H * D].view(N, H, D))
        far[-1].copy_(t)
    order = perm(N)
    both(*far, do, offs(LENS), causal=True, order=order)
    o = sp.spconv_attention(q, k, v, offs(LENS), causal=True, order=order)
    assert torch.equal(sp.spconv_attention(*far, offs(LENS), causal=True, order=order), o)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_large_and_growing_scores(dt):
    """Scores of thousands, ever larger along the keys: the reference is taken again."""
    seqs, L, D = 10, 300, 32
    q, k, v, do, _ = make(seqs * L, seqs * L, 8, 8, D, dt, 13)
    k = k * torch.linspace(1, 60, L, device="cuda").repeat(seqs)[:, None, None].to(dt)
    o = offs([L] * seqs)
    for causal in (False, True):
        call = lambda: sp.spconv_attention(q, k, v, o, scale=2.0, causal=causal, stats=True)
        assert_launches(call, f"k_attn<{NAMES[dt]}, 32>")
        want = attention64(q, k, v, o, scale=2.0, causal=causal)
        for got, name in zip(call(), ("out", "lse")):
            check(got, want[name], name)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3e38])
def test_hidden_rows_have_no_effect(dt, D, value):
    """Causal sequences of 600 rows: what later keys hold does not reach earlier
    queries' outputs and gradients, nor what earlier queries hold later keys'
    gradients, nor rows behind the sequences anything."""
    seqs, L, cut, H = 6, 600, 400, 8
    q, k, v, do, _ = make(seqs * L + 50, seqs * L + 50, H, H, D, dt, 11)
    o = offs([L] * seqs)
    what = f"<{NAMES[dt]}, {D}"
    fwd = lambda *t: sp.spconv_attention(*t, o, causal=True, stats=True)
    out, lse = fwd(q, k, v)
    grad = lambda *t: sp.spconv_attention_grad(*t, out, lse, o, causal=True)
    assert_launches(lambda: fwd(q, k, v), f"k_attn{what}>")
    assert_launches(lambda: grad(do, q, k, v), f"k_attn_dq{what}, 0>", f"k_attn_dkv{what}, 0>")
    want = grad(do, q, k, v)
    rows = lambda t: t[:seqs * L].view(seqs, L, *t.shape[1:])
    bad = lambda t, at: (rows(t)[:, at].fill_(value), t[seqs * L:].fill_(value), t)[2]
    k2, v2 = (bad(t.clone(), slice(cut, None, 7)) for t in (k, v))
    got = fwd(q, k2, v2)
    assert torch.equal(rows(got[0])[:, :cut], rows(out)[:, :cut])
    assert torch.equal(rows(got[1])[:, :cut], rows(lse)[:, :cut])
    assert torch.equal(rows(grad(do, q, k2, v2)[0])[:, :cut], rows(want[0])[:, :cut])
    q2, do2 = (bad(t.clone(), slice(0, cut, 7)) for t in (q, do))
    for a, b in zip(grad(do2, q2, k, v)[1:], want[1:]):
        assert torch.equal(rows(a)[:, cut:], rows(b)[:, cut:])


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_infinite_and_unknown_values(dt):
    """An infinite value reaches the queries that see it; a query of NaN only itself."""
    seqs, L, H, D = 10, 300, 8, 64
    q, k, v, do, _ = make(seqs * L, seqs * L, H, H, D, dt, 12)
    at = 2 * L + 150
    v[at, 0, 3] = float("inf")
    q[L + 5] = float("nan")
    call = lambda: sp.spconv_attention(q, k, v, offs([L] * seqs), causal=True, stats=True)
    assert_launches(call, f"k_attn<{NAMES[dt]}, 64>")
    out, lse = call()
    assert bool((out[at:3 * L, 0, 3] == float("inf")).all())
    assert bool(torch.isnan(out[L + 5]).all()) and bool(torch.isnan(lse[L + 5]).all())
    odd = ~torch.isfinite(out)
    assert int(odd.sum()) == 150 + H * D
    assert int((~torch.isfinite(lse)).sum()) == H


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_gradient_against_differences(dt):
    """The gradients of the kernels that share tiles, along a direction, against
    differences of the 32-bit forward's 64-bit sums."""
    g = torch.Generator().manual_seed(5)
    lens = [300] * 10
    N, H, D = sum(lens), 8, 32
    q, k, v, do = (torch.randn(N, H, D, generator=g).to(dt).cuda() for _ in range(4))
    o = offs(lens)
    out, lse = sp.spconv_attention(q, k, v, o, causal=True, stats=True)
    grads = sp.spconv_attention_grad(do, q, k, v, out, lse, o, causal=True)
    what = f"<{NAMES[dt]}, {D}, 0>"
    assert_launches(lambda: sp.spconv_attention_grad(do, q, k, v, out, lse, o, causal=True), "k_attn_dq" + what,
                    "k_attn_dkv" + what)
    f = lambda *t: float((sp.spconv_attention(*t, o, causal=True).double() * do.double()).sum())
    wide = [t.float() for t in (q, k, v)]
    for i in range(3):
        d = torch.randn(N, H, D, generator=g).cuda()
        step = 1e-2
        args = list(wide)
        args[i] = wide[i] + step * d
        hi = f(*args)
        args[i] = wide[i] - step * d
        lo = f(*args)
        want = float((grads[i].double() * d.double()).sum())
        # third-order term step^2 / 6 f''' and 32-bit outputs over 2 step; bf16 gradients are
        # off by less than 2^-8 + 2^-8 of their norm, at random signs against d
        size = float(do.double().norm()) * float(d.double().norm())
        allowed = size * (step ** 2 + 2 ** -24 * 8 / step)
        if dt == BF:
            allowed += 2 ** -7 * float(grads[i].double().norm()) * 6
        assert abs((hi - lo) / (2 * step) - want) <= allowed, i
