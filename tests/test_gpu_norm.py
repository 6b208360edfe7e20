"""Layer norm and its gradient on the GPU against their formulas in 64 bits.

Tolerances: an output in type t is rounded once (eps_t / 2 of its value); the
fp32 arithmetic before it adds u = 2^-24 for each rounding.  A row's sums run
over at most 16 elements in a lane and then log2(64) + 4 joins, so a mean is
off by at most 26 u of the mean magnitude; 32 u covers the few roundings next
to it (forward), 64 u the two means and the products of the gradient.
dweight and dbias add rows one after the other: N / 1024 in a lane, then at
most 256 groups, 64 partials and 16 slices.
"""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
EPS = 1e-5
TINY = 1e-30


def half(dt):
    return torch.finfo(dt).eps / 2


def inputs(N, C, dt, seed=0, shift=1.0):
    g = torch.Generator().manual_seed(seed * 7919 + N * 31 + C)
    x = torch.randn(N, C, generator=g) * (torch.rand(C, generator=g) + 0.5) + shift * torch.randn(C, generator=g)
    w = 1 + 0.2 * torch.randn(C, generator=g)
    b = 0.2 * torch.randn(C, generator=g)
    d = torch.randn(N, C, generator=g)
    return x.to(dt).to(DEV), w.to(DEV), b.to(DEV), d.to(dt).to(DEV)


def forward64(x, w, b, eps=EPS):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * rstd
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max()):.3g} of the tolerance"
    assert torch.isfinite(got.double()).all()


def check_forward(x, w, b, eps=EPS):
    y, mean, rstd = sp.spconv_layernorm(x, w, b, eps=eps, stats=True)
    y64, m64, r64 = forward64(x, w, b, eps)
    mag = x.double().abs().mean(1, keepdim=True)
    aw = w.double().abs() if w is not None else 1.0
    b64 = b.double() if b is not None else torch.zeros((), dtype=torch.float64, device=DEV)
    tol = half(x.dtype) * y64.abs() + 32 * U * (r64 * aw * mag + (y64 - b64).abs() + b64.abs()) + TINY
    assert y.dtype == x.dtype
    within(y, y64, tol, "y")
    within(mean, m64[:, 0], 32 * U * mag[:, 0] + TINY, "mean")
    within(rstd, r64[:, 0], 32 * U * r64[:, 0] * (1 + (r64 * mag)[:, 0] * 32 * U), "rstd")
    return y, mean, rstd


def check_grad(d, x, mean, rstd, w):
    dx, dw, db = sp.spconv_layernorm_grad(d, x, mean, rstd, w)
    N = x.shape[0]
    d64, r = d.double(), rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    g = d64 * w.double() if w is not None else d64
    dx64 = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    mag = r * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    assert dx.dtype == x.dtype
    within(dx, dx64, half(x.dtype) * dx64.abs() + 64 * U * mag + TINY, "dx")
    if w is None:
        assert dw is None and db is None
        return dx, dw, db
    chain = (N // 1024 + 340) * U
    within(dw, (d64 * xh).sum(0), chain * (d64 * xh).abs().sum(0) + TINY, "dweight")
    within(db, d64.sum(0), chain * d64.abs().sum(0) + TINY, "dbias")
    return dx, dw, db


CS = [1, 2, 3, 8, 9, 17, 31, 64, 100, 127, 128, 129, 256, 387, 511, 520, 777, 1024, 1025, 2047, 2048, 2056, 4095, 4096]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", CS)
def test_widths(C, dt):
    for N in (1, 2, 37, 600):
        x, w, b, d = inputs(N, C, dt)
        _, mean, rstd = check_forward(x, w, b)
        check_grad(d, x, mean, rstd, w)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N, C", [(40001, 128), (70003, 24), (9001, 387), (3001, 1500), (300007, 8)])
def test_many_rows(N, C, dt):
    x, w, b, d = inputs(N, C, dt)
    _, mean, rstd = check_forward(x, w, b)
    check_grad(d, x, mean, rstd, w)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_without_weight_bias_or_statistics(dt):
    x, w, b, d = inputs(77, 96, dt)
    _, mean, rstd = check_forward(x, None, None)
    check_grad(d, x, mean, rstd, None)
    check_forward(x, w, None)
    check_forward(x, None, b)
    y = sp.spconv_layernorm(x, w, b)
    assert torch.is_tensor(y) and torch.equal(y, sp.spconv_layernorm(x, w, b, stats=True)[0])


def test_far_from_zero_and_constant_rows():
    """A mean a thousand times the spread; rows without spread (eps alone)."""
    x, w, b, d = inputs(50, 200, torch.float32, shift=1000.0)
    x[7] = 3.25
    x[8] = 0
    _, mean, rstd = check_forward(x, w, b)
    assert abs(float(rstd[7]) * EPS ** 0.5 - 1) < 1e-6
    check_grad(d, x, mean, rstd, w)


def test_bad_values_stay_in_their_rows():
    x, w, b, d = inputs(40, 130, torch.bfloat16)
    y0 = sp.spconv_layernorm(x, w, b)
    x[3, 5], x[20, 129], x[21, 0] = float("nan"), float("inf"), float("-inf")
    y = sp.spconv_layernorm(x, w, b)
    rows = [3, 20, 21]
    assert torch.isnan(y[rows]).all()
    keep = [i for i in range(40) if i not in rows]
    assert torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_views_alignment_streams_and_repeats(dt):
    x, w, b, d = inputs(300, 72, dt)
    want = sp.spconv_layernorm(x, w, b, stats=True)
    grad = sp.spconv_layernorm_grad(d, x, want[1], want[2], w)
    # rows of a wider tensor, and rows that start one element into a buffer
    wide = torch.cat([x, x], 1)[:, :72]
    off = torch.empty(300 * 72 + 1, dtype=dt, device=DEV)[1:].view(300, 72).copy_(x)
    assert not wide.is_contiguous() and off.data_ptr() % 16 != 0
    for v in (wide, off):
        for a, c in zip(sp.spconv_layernorm(v, w, b, stats=True), want):
            assert torch.equal(a, c)
        for a, c in zip(sp.spconv_layernorm_grad(d, v, want[1], want[2], w), grad):
            assert torch.equal(a, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = sp.spconv_layernorm_grad(d, x, want[1], want[2], w)
    torch.cuda.current_stream().wait_stream(s)
    for a, c in zip(other, grad):
        assert torch.equal(a, c)
    # in place
    y = x.clone()
    assert sp.spconv_layernorm(y, w, b, out=y) is y and torch.equal(y, want[0])


def test_no_rows():
    x = torch.empty(0, 64, device=DEV)
    s = torch.empty(0, device=DEV)
    y, mean, rstd = sp.spconv_layernorm(x, stats=True)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = sp.spconv_layernorm_grad(x, x, s, s, torch.ones(64, device=DEV))
    assert dx.shape == (0, 64) and torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_gradient_against_differences():
    """Central differences of the 64-bit forward along random directions."""
    x, w, b, d = inputs(60, 48, torch.float32)
    _, mean, rstd = sp.spconv_layernorm(x, w, b, stats=True)
    dx, dw, db = sp.spconv_layernorm_grad(d, x, mean, rstd, w)
    d64, h = d.double(), 1e-6
    g = torch.Generator().manual_seed(3)
    for which, grad in (("x", dx), ("w", dw), ("b", db)):
        base = {"x": x.double(), "w": w.double(), "b": b.double()}
        v = torch.randn(grad.shape, generator=g).double().to(DEV)
        up, down = dict(base), dict(base)
        up[which], down[which] = base[which] + h * v, base[which] - h * v
        diff = ((forward64(up["x"], up["w"], up["b"])[0] - forward64(down["x"], down["w"], down["b"])[0]) * d64).sum()
        diff = float(diff) / (2 * h)
        # fp32 gradients: 64 u per entry against the sum of magnitudes; the difference itself is off by h^2 and 2^-53 / h
        scale = float((grad.double() * v).abs().sum())
        assert abs(float((grad.double() * v).sum()) - diff) <= 1e-5 * scale, which


def test_refuses_what_does_not_fit():
    x = torch.zeros(4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    s = torch.zeros(4, device=DEV)
    for bad in (lambda: sp.spconv_layernorm(x.half()), lambda: sp.spconv_layernorm(x, w[:32]),
                lambda: sp.spconv_layernorm(x, w.cpu()), lambda: sp.spconv_layernorm(x, w.bfloat16()),
                lambda: sp.spconv_layernorm(x, out=torch.empty(4, 32, device=DEV)),
                lambda: sp.spconv_layernorm_grad(x.bfloat16(), x, s, s, w),
                lambda: sp.spconv_layernorm_grad(x, x, s[:2], s, w),
                lambda: sp.spconv_layernorm_grad(x, x, s, None, w),
                lambda: sp.spconv_layernorm_grad(x, x, s, s, w, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sp.SpconvError) as e:
        sp.spconv_layernorm(torch.zeros(2, 4097, device=DEV))
    assert e.value.code == -2
