"""Infinite states and gradients of the recurrence on the GPU."""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DTS = pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


@DTS
@pytest.mark.parametrize("N, C", [(300, 24), (3000, 128), (9000, 128), (20000, 6)])
def test_infinite_states_stay_infinite(N, C, dt):
    """f s is infinite for every f above zero, however many of them are
    composed: states after an infinite row are infinite to the scene's end,
    step by step and in each channel, gradients before one too."""
    cut, at = N // 10, N // 5
    off = [0, cut, N]
    g = torch.Generator().manual_seed(N)
    x, d = (torch.randn(N, C, generator=g).to(dt).to(DEV) for _ in range(2))
    z = (torch.linspace(5, -40, C)[None] + torch.randn(N, C, generator=g)).to(dt).to(DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    h0 = torch.zeros(2, C, device=DEV)
    h, last = sp.spconv_scan(x, z, o, h0=h0)
    xb, db = x.clone(), d.clone()
    xb[at], db[N - 10] = float("inf"), float("-inf")
    hb, lastb = sp.spconv_scan(xb, z, o, h0=h0)
    assert torch.equal(hb[:at], h[:at]) and torch.equal(lastb[0], last[0])
    assert torch.isposinf(hb[at:]).all() and torch.isposinf(lastb[1]).all()
    h0[1] = float("-inf")
    hb, lastb = sp.spconv_scan(x, z, o, h0=h0)
    assert torch.equal(hb[:cut], h[:cut]) and torch.isneginf(hb[cut:]).all() and torch.isneginf(lastb[1]).all()
    h0[1] = 0
    dx, _, dh0 = sp.spconv_scan_grad(d, x, z, o, h0=h0)
    dxb, _, dh0b = sp.spconv_scan_grad(db, x, z, o, h0=h0)
    assert torch.equal(dxb[:cut], dx[:cut]) and torch.equal(dxb[N - 9:], dx[N - 9:]) and torch.equal(dh0b[0], dh0[0])
    assert torch.isneginf(dxb[cut:N - 9]).all() and torch.isneginf(dh0b[1]).all()


@DTS
def test_closed_gate_ends_an_infinite_state_as_a_step_does(dt):
    """A gate that is zero in 32 bits times infinity is NaN, from that row on,
    and the rows before it keep their infinity."""
    N, C, at, shut = 6000, 128, 500, 4000
    x, z = torch.ones(N, C, dtype=dt, device=DEV), torch.full((N, C), -12.0, dtype=dt, device=DEV)
    x[at], z[shut] = float("inf"), float("-inf")
    h, last = sp.spconv_scan(x, z, torch.tensor([0, N], dtype=torch.int32, device=DEV))
    assert torch.isfinite(h[:at].float()).all() and torch.isposinf(h[at:shut]).all() and torch.isnan(h[shut:]).all()
    assert torch.isnan(last).all()
