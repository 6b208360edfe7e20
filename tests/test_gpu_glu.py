"""Gated linear unit and its gradient on the GPU against their formulas in 64
bits.

Tolerances, u = 2^-24: a projection adds C products and a bias in fp32, off by
at most (C + 4) u of the summed magnitudes; an activation or its derivative by
(2 |a| + 8) u (1 + |a|) (the rounded exponent, then a few roundings) and its
slope, at most 1.2, times the projection's error.  In bfloat16 da and db are
rounded once before the products (half an eps of their value), the outputs of
either type once at the end.  Sums over F or N terms add that many u of the
summed magnitudes.  Magnitudes hide a lost row among thousands, so the
gradients are also taken with dout zero outside single rows.
"""
import math

import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
TINY = 1e-30
DTS = pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


def half(dt):
    return torch.finfo(dt).eps / 2


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, "
                           f"worst {float((err / tol).max()):.3g} of the tolerance")


def inputs(N, C, F, dt, bias, seed=0):
    g = torch.Generator().manual_seed(seed * 101 + N * 7 + C * 3 + F)
    x = torch.randn(N, C, generator=g).to(dt).to(DEV)
    w = (torch.randn(2, C, F, generator=g) * 1.5 * C ** -0.5).to(dt).to(DEV)
    b = (0.3 * torch.randn(2, F, generator=g)).to(DEV) if bias else None
    d = torch.randn(N, F, generator=g).to(dt).to(DEV)
    return x, w, b, d


def act64(a, kind):
    if kind == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    cdf = 0.5 * torch.special.erfc(-a / math.sqrt(2))
    return a * cdf, cdf + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)


def forward64(x, w, b, kind):
    """h and the pieces of its bounds."""
    x, w = x.double(), w.double()
    p = [x @ w[s] + (b[s].double() if b is not None else 0) for s in (0, 1)]
    mag = [x.abs() @ w[s].abs() + (b[s].double().abs() if b is not None else 0) for s in (0, 1)]
    e = [(x.shape[1] + 4) * U * m for m in mag]
    v, d = act64(p[0], kind)
    ev = 1.2 * e[0] + (2 * p[0].abs() + 8) * U * (1 + p[0].abs())
    return p, e, v, d, ev


def check_forward(x, w, b, kind):
    h = sp.spconv_glu(x, w, b, act=kind)
    p, e, v, _, ev = forward64(x, w, b, kind)
    want = v * p[1]
    err = ev * p[1].abs() + v.abs() * e[1] + ev * e[1] + 2 * U * want.abs()
    assert h.dtype == x.dtype
    within(h, want, half(x.dtype) * (want.abs() + err) + err + TINY, "h")


def check_grad(d, x, w, b, kind):
    dx, dw, db = sp.spconv_glu_grad(d, x, w, b, act=kind)
    N, C = x.shape
    F = w.shape[2]
    p, e, v, s, ev = forward64(x, w, b, kind)
    dh = d.double()
    r = half(torch.bfloat16) if x.dtype == torch.bfloat16 else 0.0
    g = [dh * p[1] * s, dh * v]
    eg = [dh.abs() * (p[1].abs() * ev + s.abs() * e[1] + ev * e[1]) + 3 * U * g[0].abs(), dh.abs() * ev + 2 * U * g[1].abs()]
    er = [eg[k] + r * (g[k].abs() + eg[k]) for k in (0, 1)]      # as operands
    x64, w64 = x.double(), w.double()
    want = g[0] @ w64[0].t().contiguous() + g[1] @ w64[1].t().contiguous()
    mag = sum(g[k].abs() @ w64[k].abs().t().contiguous() for k in (0, 1))
    err = sum(er[k] @ w64[k].abs().t().contiguous() for k in (0, 1)) + (2 * F + 4) * U * mag
    within(dx, want, half(x.dtype) * (want.abs() + err) + err + TINY, "dx")
    xt = x64.t().contiguous()
    rows = int((dh.abs().sum(1) > 0).sum()) + 8
    for k in (0, 1):
        want = xt @ g[k]
        err = xt.abs() @ er[k] + rows * U * (xt.abs() @ g[k].abs())
        within(dw[k], want, half(x.dtype) * (want.abs() + err) + err + TINY, f"dw[{k}]")
        if b is not None:
            err = eg[k].sum(0) + rows * U * g[k].abs().sum(0)
            within(db[k], g[k].sum(0), err + U * g[k].sum(0).abs() + TINY, f"dbias[{k}]")
    assert dx.dtype == x.dtype and dw.dtype == x.dtype and (db is None) == (b is None)


SHAPES = [(1, 8, 8), (1, 256, 1024), (2, 128, 256), (3, 40, 24), (16, 64, 168), (17, 72, 8), (33, 8, 640), (63, 128, 64),
          (64, 256, 72), (65, 32, 256), (127, 136, 136), (128, 128, 128), (129, 128, 256), (200, 1024, 48),
          (255, 16, 1000), (300, 264, 520), (513, 96, 96), (1025, 128, 256), (40, 4096, 16), (40, 16, 4096)]


@DTS
@pytest.mark.parametrize("N, C, F", SHAPES)
def test_shapes(N, C, F, dt):
    for kind, bias in (("silu", True), ("gelu", False)):
        x, w, b, d = inputs(N, C, F, dt, bias)
        check_forward(x, w, b, kind)
        check_grad(d, x, w, b, kind)


@DTS
@pytest.mark.parametrize("N, C, F", [(20000, 128, 256), (9001, 256, 680), (30001, 64, 168), (70001, 24, 40), (5000, 512, 136)])
def test_many_rows(N, C, F, dt):
    x, w, b, d = inputs(N, C, F, dt, True)
    check_forward(x, w, b, "gelu")
    check_grad(d, x, w, b, "silu")


@DTS
@pytest.mark.parametrize("N, C, F", [(5, 72, 1544), (130, 200, 2008), (1, 1024, 4096), (700, 64, 840), (260, 8, 392), (2100, 40, 1000)])
def test_few_rows_of_wide_weights(N, C, F, dt):
    """The input gradient's reduction in splits, which end inside the halves."""
    for kind, bias in (("silu", False), ("gelu", True)):
        x, w, b, d = inputs(N, C, F, dt, bias)
        check_grad(d, x, w, b, kind)


@pytest.mark.parametrize("N, C, F", [(32768, 128, 256), (40007, 128, 264), (33000, 8, 8), (50001, 40, 1000),
                                     (66000, 64, 72), (65537, 104, 512), (100003, 24, 136), (33333, 96, 2048)])
def test_rows_with_few_channels(N, C, F):
    """bfloat16 with many rows: weights kept on the chip, in one slab or several."""
    for kind, bias in (("silu", True), ("gelu", False)):
        x, w, b, d = inputs(N, C, F, torch.bfloat16, bias)
        check_forward(x, w, b, kind)
        check_grad(d, x, w, b, kind)
    for r in (0, 17, 63, 64, 255, 256, 8191, 32767, N - 1):
        one = torch.zeros_like(d)
        one[r] = d[r]
        check_grad(one, x, w, b, "silu")


@DTS
@pytest.mark.parametrize("N, C, F", [(3000, 128, 256), (3001, 64, 168), (2500, 256, 680), (2049, 40, 24)])
def test_single_rows(N, C, F, dt):
    """dout is zero outside one row: its dw, dbias and dx alone."""
    x, w, b, d = inputs(N, C, F, dt, True)
    for r in (0, 1, 15, 16, 31, 63, 64, 127, 128, 511, 512, 1023, 2047, N - 1):
        one = torch.zeros_like(d)
        one[r] = d[r]
        check_grad(one, x, w, b, "silu")


@DTS
def test_weights_that_pick_single_entries(dt):
    """w with one entry: h has one column, dx one channel, so a wrong index
    shows whatever the sums."""
    N, C, F = 130, 136, 200
    x, _, _, d = inputs(N, C, F, dt, False)
    for c, f in ((0, 0), (7, 8), (31, 63), (32, 64), (127, 127), (128, 128), (135, 199)):
        w = torch.zeros(2, C, F, dtype=dt, device=DEV)
        w[0, c, f], w[1, c, f] = 1.5, -0.75
        check_forward(x, w, None, "silu")
        check_grad(d, x, w, None, "gelu")


@DTS
def test_bad_values_stay_in_their_rows(dt):
    x, w, b, d = inputs(300, 64, 72, dt, True)
    h0 = sp.spconv_glu(x, w, b)
    dx0 = sp.spconv_glu_grad(d, x, w, b)[0]
    xb, db = x.clone(), d.clone()
    xb[5, 3], xb[130, 60], db[200, 7] = float("nan"), float("inf"), float("nan")
    h = sp.spconv_glu(xb, w, b)
    dx = sp.spconv_glu_grad(db, xb, w, b)[0]
    keep = [i for i in range(300) if i not in (5, 130, 200)]
    assert torch.equal(h[keep], h0[keep]) and torch.equal(dx[keep], dx0[keep])
    assert torch.isnan(h[5]).all() and not torch.isfinite(h[130].float()).all() and torch.equal(h[200], h0[200])
    assert torch.isnan(dx[5]).all() and torch.isnan(dx[200]).all()


@DTS
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_large_arguments(kind, dt):
    """Projections far outside the exponential's range: act(a) is a or 0."""
    x = torch.full((4, 8), 16.0, dtype=dt, device=DEV)
    w = torch.zeros(2, 8, 16, dtype=dt, device=DEV)
    w[0, :, :8], w[0, :, 8:], w[1] = 16.0, -16.0, 0.0078125
    h = sp.spconv_glu(x, w, act=kind)
    assert torch.equal(h[:, :8], torch.full_like(h[:, :8], 2048.0)) and torch.count_nonzero(h[:, 8:]) == 0
    dx, dw, _ = sp.spconv_glu_grad(torch.ones_like(h), x, w, act=kind)
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dw.float()).all()


@DTS
def test_views_streams_and_repeats(dt):
    x, w, b, d = inputs(1000, 64, 128, dt, True)
    f = lambda x, w, d: (sp.spconv_glu(x, w, b), *sp.spconv_glu_grad(d, x, w, b))
    want = f(x, w, d)
    wide = [torch.cat([t, t], -1)[..., :t.shape[-1]] for t in (x, w, d)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = f(x, w, d)
    torch.cuda.current_stream().wait_stream(st)
    for got in (f(*wide), f(x, w, d), other):
        for a, c in zip(got, want):
            assert torch.equal(a, c)


def test_no_rows():
    x = torch.empty(0, 64, device=DEV)
    w = torch.ones(2, 64, 32, device=DEV)
    b = torch.ones(2, 32, device=DEV)
    assert sp.spconv_glu(x, w, b).shape == (0, 32)
    dx, dw, db = sp.spconv_glu_grad(torch.empty(0, 32, device=DEV), x, w, b)
    assert dx.shape == (0, 64) and torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradient_against_differences(kind):
    x, w, b, d = inputs(50, 24, 32, torch.float32, True)
    grads = [t.double() for t in sp.spconv_glu_grad(d, x, w, b, act=kind)]
    base, h = [x.double(), w.double(), b.double()], 1e-6

    def loss(x, w, b):
        return float((act64(x @ w[0] + b[0], kind)[0] * (x @ w[1] + b[1]) * d.double()).sum())

    g = torch.Generator().manual_seed(4)
    for k, grad in enumerate(grads):
        v = torch.randn(grad.shape, generator=g).double().to(DEV)
        up, down = list(base), list(base)
        up[k], down[k] = base[k] + h * v, base[k] - h * v
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # fp32 gradients: about 100 u of the summed magnitudes; differences: h^2 and 2^-53 / h
        assert abs(float((grad * v).sum()) - diff) <= 1e-5 * float((grad * v).abs().sum()), k


def test_refuses_what_does_not_fit():
    x = torch.zeros(4, 64, device=DEV)
    w = torch.zeros(2, 64, 32, device=DEV)
    d = torch.zeros(4, 32, device=DEV)
    for bad in (lambda: sp.spconv_glu(x, w.bfloat16()), lambda: sp.spconv_glu(x, w[:1]), lambda: sp.spconv_glu(x, w[:, :32]),
                lambda: sp.spconv_glu(x, w.cpu()), lambda: sp.spconv_glu(x, w, act="relu"),
                lambda: sp.spconv_glu(x, w, torch.zeros(32, device=DEV)), lambda: sp.spconv_glu(x.half(), w.half()),
                lambda: sp.spconv_glu_grad(x, x, w), lambda: sp.spconv_glu_grad(None, x, w),
                lambda: sp.spconv_glu_grad(d, x, w, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for C, F in ((60, 32), (64, 36), (4104, 8), (8, 4104)):
        with pytest.raises(sp.SpconvError) as e:
            sp.spconv_glu(torch.zeros(2, C, device=DEV), torch.zeros(2, C, F, device=DEV))
        assert e.value.code == -2
