"""Which of the layer norm's sums over rows a gradient returns.

Tolerances: u = 2^-24; dweight and dbias add N rows, each product rounded once
or twice: (N + 4) u of the summed magnitudes.
"""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N, C", [(0, 24), (1, 8), (77, 96), (700, 387), (30, 4096)])
def test_bias_without_weight(N, C, dt):
    g = torch.Generator().manual_seed(N + C)
    x, d = (torch.randn(N, C, generator=g).to(dt).to(DEV) for _ in range(2))
    b = torch.randn(C, generator=g).to(DEV)
    _, mean, rstd = sp.spconv_layernorm(x, None, b, stats=True)
    dx, dw, db = sp.spconv_layernorm_grad(d, x, mean, rstd, sums=True)
    plain = sp.spconv_layernorm_grad(d, x, mean, rstd)
    assert torch.equal(dx, plain[0]) and plain[1] is None and plain[2] is None
    one = sp.spconv_layernorm_grad(d, x, mean, rstd, torch.ones(C, device=DEV))
    assert torch.equal(dx, one[0]) and torch.equal(dw, one[1]) and torch.equal(db, one[2])
    d64 = d.double()
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got, t in ((dw, d64 * xh), (db, d64)):
        assert got.dtype == torch.float32
        assert ((got.double() - t.sum(0)).abs() <= (N + 4) * U * t.abs().sum(0)).all()


def test_gradient_of_x_alone():
    x = torch.randn(50, 40, device=DEV)
    w = torch.rand(40, device=DEV)
    _, mean, rstd = sp.spconv_layernorm(x, w, stats=True)
    dx, dw, db = sp.spconv_layernorm_grad(x, x, mean, rstd, w, sums=False)
    assert dw is None and db is None
    assert torch.equal(dx, sp.spconv_layernorm_grad(x, x, mean, rstd, w)[0])
