"""Gated recurrence and its gradient on the GPU against the recurrence walked
step by step in 64 bits.

Tolerances: the reference walks a bound next to each value.  With u = 2^-24 a
gate's exponent is off by 2 u |z| (the rounded product with log2 e), the
exponential, the reciprocal, the sums and products by at most 10 u more, so a
step adds c u times the magnitude of the state, c = 2 |z| + 10, and earlier
errors decay with f like the state does: E[t] = f E[t-1] + c u H[t], H the
recurrence over magnitudes.  Composing steps into maps rounds the same
products, once each.  The output's type adds eps / 2 of the value.
"""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
TINY = 1e-30


def half(dt):
    return torch.finfo(dt).eps / 2


def within(got, want, tol, what):
    got = got.double().cpu()
    err = (got - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at "
                           f"{bad.nonzero()[0].tolist()}, worst {float((err / tol).max()):.3g} of the tolerance")


def walk(x, z, off, order, h0, dout=None, dlast=None):
    """Values and error bounds, in 64 bits on the host, rows in the caller's order."""
    x, z = x.double().cpu(), z.double().cpu()
    N, C = x.shape
    B = len(off) - 1
    rows = order.cpu().long().tolist() if order is not None else list(range(N))
    f, n, c = torch.sigmoid(z), torch.sigmoid(-z), (2 * z.abs() + 10) * U
    h, H, E = (torch.zeros(N, C, dtype=torch.float64) for _ in range(3))
    prev, prevH, prevE = (torch.zeros(N, C, dtype=torch.float64) for _ in range(3))
    last, lastE = torch.zeros(B, C, dtype=torch.float64), torch.zeros(B, C, dtype=torch.float64)
    for b in range(B):
        s = h0[b].double().cpu() if h0 is not None else torch.zeros(C, dtype=torch.float64)
        a, e = s.abs(), torch.zeros(C, dtype=torch.float64)
        for t in range(off[b], off[b + 1]):
            r = rows[t]
            prev[r], prevH[r], prevE[r] = s, a, e
            s = f[r] * s + n[r] * x[r]
            a = f[r] * a + n[r] * x[r].abs()
            e = f[r] * e + c[r] * a
            h[r], H[r], E[r] = s, a, e
        last[b], lastE[b] = s, e
    out = {"h": (h, E), "last": (last, lastE)}
    if dout is None:
        return out
    d = dout.double().cpu()
    g, G, Eg = (torch.zeros(N, C, dtype=torch.float64) for _ in range(3))
    dh0, dh0E = torch.zeros(B, C, dtype=torch.float64), torch.zeros(B, C, dtype=torch.float64)
    for b in range(B):
        y = dlast[b].double().cpu() if dlast is not None else torch.zeros(C, dtype=torch.float64)
        a, e = y.abs(), torch.zeros(C, dtype=torch.float64)
        for t in reversed(range(off[b], off[b + 1])):
            r = rows[t]
            g[r] = d[r] + y
            G[r] = d[r].abs() + a
            Eg[r] = e + 2 * U * G[r]
            y, a, e = f[r] * g[r], f[r] * G[r], f[r] * Eg[r] + c[r] * f[r] * G[r]
        dh0[b], dh0E[b] = y, e
    w = (prev - x)
    W = prevH + x.abs()
    out["dx"] = (n * g, n * (Eg + c * G))
    out["dz"] = (g * w * f * n, f * n * (Eg * W + G * prevE + (3 * c + 4 * U) * G * W))
    out["dh0"] = (dh0, dh0E)
    return out


def inputs(N, C, dt, off, order, h0, seed=0):
    g = torch.Generator().manual_seed(seed * 977 + N * 13 + C)
    B = len(off) - 1
    reach = torch.rand(C, generator=g) * 6 + 1
    x = torch.randn(N, C, generator=g).to(dt).to(DEV)
    z = (torch.randn(N, C, generator=g) * 1.5 + reach).to(dt).to(DEV)
    d = torch.randn(N, C, generator=g).to(dt).to(DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    perm = torch.randperm(N, generator=g).to(torch.int32).to(DEV) if order else None
    s = torch.randn(B, C, generator=g).to(DEV) if h0 else None
    dl = torch.randn(B, C, generator=g).to(DEV)
    return x, z, d, o, perm, s, dl


def check(N, C, dt, off, order=False, h0=False, seed=0):
    x, z, d, o, perm, s, dl = inputs(N, C, dt, off, order, h0, seed)
    want = walk(x, z, off, perm, s, d, dl)
    h, last = sp.spconv_scan(x, z, o, order=perm, h0=s)
    dx, dz, dh0 = sp.spconv_scan_grad(d, x, z, o, order=perm, h0=s, dlast=dl)
    assert h.dtype == dt and dx.dtype == dt and dz.dtype == dt and last.dtype == torch.float32
    for name, got in (("h", h), ("dx", dx), ("dz", dz)):
        v, e = want[name]
        within(got, v, half(dt) * v.abs() + e * (1 + half(dt)) + TINY, name)
    within(last, want["last"][0], want["last"][1] + U * want["last"][0].abs() + TINY, "last")
    if h0:
        within(dh0, want["dh0"][0], want["dh0"][1] + U * want["dh0"][0].abs() + TINY, "dh0")
    else:
        assert dh0 is None


DTS = pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


@DTS
@pytest.mark.parametrize("C", [1, 3, 4, 8, 9, 16, 31, 32, 64, 65, 100, 128, 136, 257])
def test_widths(C, dt):
    check(700, C, dt, [0, 130, 131, 700], order=True, h0=True)
    check(5, C, dt, [0, 5], order=False, h0=False)


@DTS
@pytest.mark.parametrize("N", [1, 2, 7, 8, 63, 64, 65, 127, 128, 129, 255, 256, 257, 2047, 2048, 2049, 4500])
def test_lengths(N, dt):
    check(N, 40, dt, [0, N], order=False, h0=True)
    check(N, 40, dt, [0, N // 3, N], order=True, h0=False)


@DTS
def test_scenes(dt):
    """Empty scenes in front, between and behind; scenes of one voxel; borders
    on chunk borders; more scenes than a workgroup has lanes."""
    check(600, 24, dt, [0, 0, 0, 1, 2, 2, 128, 256, 256, 257, 600, 600], order=True, h0=True)
    check(600, 128, dt, [0, 64, 128, 256, 512, 600], order=False, h0=True)
    check(1500, 8, dt, list(range(1501)), order=True, h0=True)
    off = sorted([0, 1700] + [(i * 37) % 1700 for i in range(1400)])
    check(1700, 17, dt, off, order=True, h0=True)


@DTS
def test_many_chunks_and_wide_rows(dt):
    check(9000, 128, dt, [0, 2000, 8999, 9000], order=True, h0=False)
    check(300, 1100, dt, [0, 300], order=False, h0=True)
    check(130, 4096, dt, [0, 70, 130], order=True, h0=True)


@DTS
@pytest.mark.parametrize("C", [1021, 1024])
def test_long_and_wide(C, dt):
    """Enough chunks for the most rows per lane, tiles of channels side by side."""
    check(8200, C, dt, [0, 0, 5000, 5001, 8200], order=True, h0=True)


@DTS
@pytest.mark.parametrize("C", [1, 2, 3, 5, 6, 7, 11, 130])
def test_row_ends(C, dt):
    """Rows that are no multiple of four channels, with scenes' states, and many
    scenes without rows around and between."""
    off = [0] * 70 + [3] * 9 + [40] + [41] * 100 + [90, 90]
    check(90, C, dt, off, order=True, h0=True)


def test_no_rows():
    x = torch.empty(0, 16, device=DEV)
    o = torch.zeros(4, dtype=torch.int32, device=DEV)
    h0 = torch.randn(3, 16, device=DEV)
    h, last = sp.spconv_scan(x, x, o, h0=h0)
    assert h.shape == (0, 16) and torch.equal(last, h0)
    assert torch.count_nonzero(sp.spconv_scan(x, x, o)[1]) == 0
    dl = torch.randn(3, 16, device=DEV)
    dx, dz, dh0 = sp.spconv_scan_grad(x, x, x, o, h0=h0, dlast=dl)
    assert dx.shape == (0, 16) and dz.shape == (0, 16) and torch.equal(dh0, dl)


@DTS
def test_closed_and_open_gates(dt):
    """z = +inf keeps the state, z = -inf replaces it, exactly; so do gates
    beyond the exponential's range."""
    N, C = 400, 20
    x, z, d, o, _, s, dl = inputs(N, C, dt, [0, N], False, True)
    for v in (float("inf"), 3e4):
        h, last = sp.spconv_scan(x, torch.full_like(z, v), o, h0=s)
        assert torch.equal(h, s.to(dt).expand(N, C)) and torch.equal(last, s)
        h, last = sp.spconv_scan(x, torch.full_like(z, -v), o, h0=s)
        assert torch.equal(h, x) and torch.equal(last[0], x[-1].float())
    dx, dz, dh0 = sp.spconv_scan_grad(d, x, torch.full_like(z, float("-inf")), o, h0=s, dlast=dl)
    assert torch.equal(dx[:-1], d[:-1]) and torch.count_nonzero(dz) == 0 and torch.count_nonzero(dh0) == 0


@DTS
def test_bad_values_stay_in_their_scene_and_channel(dt):
    N, C, off = 900, 24, [0, 300, 301, 620, 900]
    x, z, d, o, _, s, dl = inputs(N, C, dt, off, False, True)
    good = (*sp.spconv_scan(x, z, o, h0=s), *sp.spconv_scan_grad(d, x, z, o, h0=s, dlast=dl))
    xb, zb, db = x.clone(), z.clone(), d.clone()
    xb[310, 3], xb[320, 4], zb[330, 5], db[340, 6] = float("nan"), float("inf"), float("nan"), float("-inf")
    bad = (*sp.spconv_scan(xb, zb, o, h0=s), *sp.spconv_scan_grad(db, xb, zb, o, h0=s, dlast=dl))
    others = torch.ones(N, C, dtype=torch.bool, device=DEV)
    others[301:620, 3:7] = False
    states = torch.ones(4, C, dtype=torch.bool, device=DEV)
    states[2, 3:7] = False
    for a, b in zip(good, bad):
        keep = others if a.shape[0] == N else states
        assert torch.equal(a[keep], b[keep])
    h, last = bad[0], bad[1]
    assert torch.isnan(h[310:620, 3]).all() and torch.isinf(h[320:620, 4]).any() and torch.isnan(h[330:620, 5]).all()
    assert torch.isfinite(h[301:310, 3].float()).all() and not torch.isfinite(last[2, 3:6]).any()


@DTS
def test_views_alignment_streams_and_repeats(dt):
    N, C = 3000, 24
    x, z, d, o, perm, s, dl = inputs(N, C, dt, [0, 1000, N], True, True)
    f = lambda x, z, d: (*sp.spconv_scan(x, z, o, order=perm, h0=s),
                         *sp.spconv_scan_grad(d, x, z, o, order=perm, h0=s, dlast=dl))
    want = f(x, z, d)
    wide = [torch.cat([t, t], 1)[:, :C] for t in (x, z, d)]
    off = [torch.empty(N * C + 1, dtype=dt, device=DEV)[1:].view(N, C).copy_(t) for t in (x, z, d)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = f(x, z, d)
    torch.cuda.current_stream().wait_stream(st)
    for got in (f(*wide), f(*off), f(x, z, d), other):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_bad_offsets_and_order_stay_inside():
    """Wrong contents give wrong states, and touch nothing else."""
    N, C = 700, 16
    x, z, d, o, perm, s, dl = inputs(N, C, torch.float32, [0, 300, N], True, True)
    guard = torch.full((3 * N, C), 7.0, device=DEV)
    out = guard[N:2 * N]
    for off in ([5, 300, N + 900], [-40, 900, 20], [N, N, 0], [2 ** 31 - 1, -2 ** 31, 3]):
        bad = torch.tensor(off, dtype=torch.int32, device=DEV)
        sp.spconv_scan(x, z, bad, order=perm, h0=s, out=out)
        sp.spconv_scan_grad(d, x, z, bad, order=perm, h0=s, dlast=dl)
    p = perm.clone()
    p[10], p[20], p[699] = -1, N, 2 ** 31 - 1
    sp.spconv_scan(x, z, o, order=p, h0=s, out=out)
    sp.spconv_scan_grad(d, x, z, o, order=p, h0=s, dlast=dl)
    torch.cuda.synchronize()
    assert (guard[:N] == 7).all() and (guard[2 * N:] == 7).all()


def test_gradient_against_differences():
    N, C, off = 150, 6, [0, 40, 40, 150]
    x, z, d, o, perm, s, dl = inputs(N, C, torch.float32, off, True, True)
    dx, dz, dh0 = (t.double().cpu() for t in sp.spconv_scan_grad(d, x, z, o, order=perm, h0=s, dlast=dl))
    d64, dl64, h = d.double().cpu(), dl.double().cpu(), 1e-6

    def loss(x, z, s):
        w = walk(x, z, off, perm, s)
        return float((w["h"][0] * d64).sum() + (w["last"][0] * dl64).sum())

    base = [x.double(), z.double(), s.double()]
    g = torch.Generator().manual_seed(9)
    for k, grad in enumerate((dx, dz, dh0)):
        v = torch.randn(grad.shape, generator=g).double()
        up, down = list(base), list(base)
        up[k], down[k] = base[k] + h * v.to(DEV), base[k] - h * v.to(DEV)
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # fp32 gradients: (2 |z| + 10) u of the summed magnitudes along a scene; differences: h^2 and 2^-53 / h
        assert abs(float((grad * v).sum()) - diff) <= 1e-4 * float((grad * v).abs().sum()), k


def test_refuses_what_does_not_fit():
    x = torch.zeros(4, 8, device=DEV)
    o = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for bad in (lambda: sp.spconv_scan(x, x.bfloat16(), o), lambda: sp.spconv_scan(x, x, o.long()),
                lambda: sp.spconv_scan(x, x, o.cpu()), lambda: sp.spconv_scan(x, x, o[:1]),
                lambda: sp.spconv_scan(x, x, o, order=o), lambda: sp.spconv_scan(x, x, o, h0=x),
                lambda: sp.spconv_scan(x, None, o), lambda: sp.spconv_scan_grad(None, x, x, o),
                lambda: sp.spconv_scan_grad(x, x, x, o, dlast=x),
                lambda: sp.spconv_scan(x, x, o, out=torch.empty(4, 4, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sp.SpconvError) as e:
        w = torch.zeros(2, 4097, device=DEV)
        sp.spconv_scan(w, w, o)
    assert e.value.code == -2
