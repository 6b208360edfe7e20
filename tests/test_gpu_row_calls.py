"""How the row operators' Python calls find their stream."""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu


class Without:
    """A module without some of its names."""

    def __init__(self, module, *names):
        self._module, self._names = module, names

    def __getattr__(self, name):
        if name in self._names:
            raise AttributeError(name)
        return getattr(self._module, name)


def test_torch_without_its_short_cuts(monkeypatch):
    """The public functions stand in, and give the current stream, not the
    default one."""
    x = torch.randn(3000, 128, device="cuda")
    want = sp.spconv_layernorm(x)
    with monkeypatch.context() as m:
        m.setattr(torch, "_C", Without(torch._C, "_cuda_getDevice", "_cuda_getCurrentRawStream"))
        sp._load_torch()
    try:
        assert sp._current_device is torch.cuda.current_device
        side = torch.cuda.Stream()
        assert sp._raw_stream(0) == torch.cuda.current_stream().cuda_stream
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            assert sp._raw_stream(0) == side.cuda_stream
            got = sp.spconv_layernorm(x)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
    finally:
        sp._load_torch()
    assert sp._raw_stream(0) == torch.cuda.current_stream().cuda_stream
