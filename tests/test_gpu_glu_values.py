"""The gated linear unit's activations at chosen arguments, against 64 bits.

The first channel (fp32) or the first two (bfloat16: the value's upper and
lower bits) of x are one and the others zero, so that the gate of each feature
is a value that the weights spell out, exactly; the values' weights are zero
and their bias one.  With u = 2^-24, q = P(X > |a|) and phi the normal
density, what the kernels round:

  silu  s = 1 / (1 + e), e = 2^(-a log2 e).  The exponent is off by 2 u of
        itself, which is 2 |a| u of e, the exponential by 2 u: e (2 |a| + 2) u;
        1 + e and the reciprocal add 3 u.  So ds = s (1 - s) (2 |a| + 2) u +
        3 u s, and 0 from a = 17.4 on, where 1 + e is 1 and so is its
        reciprocal.  value: |a| ds + u; slope s + a s (1 - s): its derivative
        by s is 1 + a (1 - 2 s); its own roundings are 4 u of the terms.
  gelu  q from one exponential of a^2: exponent off by 3 u of a^2 / 2, the
        polynomial in 1 / (1 + p x) and its argument by at most 32 u: q (2 a^2 +
        32) u; 1 - q rounds once.  The density: phi (2 a^2 + 8) u.  In bfloat16
        q comes from a shorter polynomial, off by 1.5e-7 / 2.
"""
import ctypes
import math

import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
TINY = 1e-36                    # below the smallest normal number the parts vanish
F32, BF16 = torch.float32, torch.bfloat16
LARGE = [0.5, 1.25, 3.0, 9.0, 12.5, 16.0, 17.0, 30.0, 1000.25, 1e5, 2.0 ** 24 + 2, 2.0 ** 25, 1e8, 3e9, 1e30]


def half(dt):
    return torch.finfo(dt).eps / 2


def gates(values, C, dt):
    """w[0] (C, F) whose column f sums, in fp32 and exactly, to a value near
    values[f], and those values in 64 bits."""
    v = torch.tensor(values, dtype=torch.float64).float()
    w = torch.zeros(C, len(values))
    w[0] = v.to(dt).float()
    if dt == BF16:
        w[1] = (v - w[0]).to(dt).float()
    a = w.double().sum(0)
    assert torch.equal(a.float().double(), a)
    return w.to(dt), a


def problem(values, N, C, dt):
    pad = -len(values) % 8
    w0, a = gates(values + [0.0] * pad, C, dt)
    w = torch.stack([w0, torch.zeros_like(w0)]).to(DEV)
    x = torch.zeros(N, C, dtype=dt, device=DEV)
    x[:, :2 if dt == BF16 else 1] = 1.0
    b = torch.zeros(2, w.shape[2], device=DEV)
    b[1] = 1.0
    return x, w, b, a


def act64(a, kind, dt):
    """Value and slope, and how far the kernels' may be off."""
    if kind == "silu":
        s, n = torch.sigmoid(a), torch.sigmoid(-a)
        v, d = a * s, s + a * s * n
        ds = torch.where(a < 17.4, s * n * (2 * a.abs() + 2) * U + 3 * U * s, 0.0)
        return v, d, a.abs() * ds + U * v.abs(), ds * (1 + a.abs() * (n - s).abs()) + 4 * U * (s + v.abs() * n)
    q = 0.5 * torch.special.erfc(a.abs() / math.sqrt(2))
    phi = torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    cdf = torch.where(a < 0, q, 1 - q)
    eq = q * (2 * a * a + 32) * U + (1.5e-7 / 2 if dt == BF16 else 0.0)
    ec = torch.where(a < 0, eq, eq + U)
    return a * cdf, cdf + a * phi, a.abs() * ec + U * (a * cdf).abs(), ec + a.abs() * phi * (2 * a * a + 8) * U + 2 * U * (
        cdf + (a * phi).abs())


def within(got, want, tol, what, values):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: at {[float(t) for t in values[bad]][:6]} got {got.double().cpu()[bad][:6].tolist()} "
                           f"for {want[bad][:6].tolist()}, worst {float((err / tol).max()):.3g} of the tolerance")


# rows and channels: tiles, bfloat16 rows with their weights on the chip, wider rows
SIZES = [(F32, 5, 8), (F32, 1000, 72), (BF16, 5, 8), (BF16, 1000, 136), (BF16, 66000, 40), (BF16, 66000, 128)]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dt, N, C", SIZES)
def test_far_arguments(dt, N, C, kind):
    """Both signs, from small to where 1 is lost next to the argument: h, dw,
    dbias, and dx with dout in one column at a time."""
    x, w, b, a = problem(LARGE + [-t for t in LARGE], N, C, dt)
    v, s, ev, es = act64(a, kind, dt)
    h = sp.spconv_glu(x, w, b, act=kind)
    for n in (0, N // 2, N - 1):
        within(h[n], v, half(dt) * (v.abs() + ev) + ev + TINY, f"h[{n}]", a)
    d = torch.zeros(N, w.shape[2], dtype=dt, device=DEV)
    d[N // 3] = 0.75
    dx, dw, db = sp.spconv_glu_grad(d, x, w, b, act=kind)
    r = half(BF16) if dt == BF16 else 0.0               # da as an operand
    da, eda = 0.75 * s, 0.75 * es + 2 * U * s.abs()
    dbv, edb = 0.75 * v, 0.75 * ev + U * v.abs()
    for k, (g, e) in enumerate(((da, eda), (dbv, edb))):
        eo = e + r * (g.abs() + e)
        within(dw[k, 0], g, half(dt) * (g.abs() + eo) + eo + TINY, f"dw[{k}]", a)
        within(db[k], g, e + U * g.abs() + TINY, f"dbias[{k}]", a)
    assert torch.count_nonzero(dw[:, 2:]) == 0
    w64 = w[0].double().cpu()
    for f in range(w.shape[2]):
        one = torch.zeros_like(d)
        one[N // 3, f] = 0.75
        dx = sp.spconv_glu_grad(one, x, w, b, act=kind)[0]
        eo = eda[f] + r * (da[f].abs() + eda[f])
        want = da[f] * w64[:, f]
        err = eo * w64[:, f].abs() + 2 * U * want.abs()
        within(dx[N // 3], want, half(dt) * (want.abs() + err) + err + TINY, "dx", a[f].expand(C))
        assert torch.count_nonzero(dx[:N // 3]) == 0 and torch.count_nonzero(dx[N // 3 + 1:]) == 0


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("N", [1, 70])
def test_single_precision_follows_the_tail(N, kind):
    """fp32 from -12 to 12: relative precision where the value is small."""
    a = torch.linspace(-12, 12, 4096).tolist()
    x, w, b, a = problem(a, N, 8, F32)
    v, s, ev, es = act64(a, kind, F32)
    h = sp.spconv_glu(x, w, b, act=kind)
    within(h[N - 1], v, ev + U * v.abs() + TINY, "h", a)
    d = torch.zeros(N, 4096, device=DEV)
    d[N - 1] = 1.0
    dw, db = sp.spconv_glu_grad(d, x, w, b, act=kind)[1:]
    for k, (g, e) in enumerate(((s, es), (v, ev))):
        within(dw[k, 0], g, e + 2 * U * g.abs() + TINY, f"dw[{k}]", a)
        within(db[k], g, e + 2 * U * g.abs() + TINY, f"dbias[{k}]", a)


@pytest.mark.parametrize("dt, N, C, F", [(F32, 3, 16, 24), (F32, 300, 16, 24), (BF16, 700, 136, 72), (BF16, 33000, 32, 40),
                                         (F32, 0, 16, 24)])
def test_bias_gradient_inside_a_packed_buffer(dt, N, C, F):
    """The C entry point takes bias and dbias at any element of a buffer, in
    calls of one tile of rows, of several, of many rows, and of none."""
    g = torch.Generator().manual_seed(N)
    x, d = torch.randn(N, C, generator=g).to(dt).to(DEV), torch.randn(N, F, generator=g).to(dt).to(DEV)
    w, b = (torch.randn(2, C, F, generator=g) / 8).to(dt).to(DEV), torch.randn(2, F, generator=g).to(DEV)
    want = sp.spconv_glu_grad(d, x, w, b)
    code = sp.SPCONV_BF16 if dt == BF16 else sp.SPCONV_F32
    n = sp.spconv_glu_grad_workspace_size(N, C, F, code)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    for at in (1, 2, 3):
        packed = torch.full((2, 2 * F + 8), 7.0, device=DEV)
        packed[0, at:at + 2 * F] = b.reshape(-1)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        rc = sp.load_library().spconv_glu_grad(p(d), p(x), p(w), p(packed[0, at:]), p(ws), n, p(dx), p(dw),
                                               p(packed[1, at:]), N, C, F, sp.SPCONV_SILU, code,
                                               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        assert torch.equal(packed[1, at:at + 2 * F], want[2].reshape(-1))
        assert (packed[1, :at] == 7).all() and (packed[1, at + 2 * F:] == 7).all()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_refuses_rows_between_16_byte_addresses(dt):
    """Contiguous views one element into a buffer, as the convolution does; a
    view that is copied (not contiguous) is taken wherever it starts."""
    x, w, d = (torch.zeros(s, dtype=dt, device=DEV) for s in ((4, 16), (2, 16, 24), (4, 24)))

    def moved(t):
        return torch.zeros(t.numel() + 1, dtype=dt, device=DEV)[1:].view(t.shape)

    for bad in (lambda: sp.spconv_glu(moved(x), w), lambda: sp.spconv_glu(x, moved(w)), lambda: sp.spconv_glu(x, w, out=moved(d)),
                lambda: sp.spconv_glu_grad(moved(d), x, w), lambda: sp.spconv_glu_grad(d, moved(x), w),
                lambda: sp.spconv_glu_grad(d, x, moved(w))):
        with pytest.raises(sp.SpconvError) as e:
            bad()
        assert e.value.code == -1 and "16-byte" in str(e.value)
    wide = torch.zeros(4, 17, dtype=dt, device=DEV)[:, 1:]
    assert wide.data_ptr() % 16 and sp.spconv_glu(wide, w).shape == (4, 24)
