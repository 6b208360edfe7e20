"""Frequencies of rotary positions (host only)."""
import math

import pytest

import submanifold_sparse_convolution_spconv_amd as sp


def freqs(*a, **k):
    return sp.spconv_rotary_freqs(*a, device="cpu", **k).tolist()


def test_axes_and_base():
    f = freqs(15, 3, base=100.0)
    assert f[:5] == f[5:10] == f[10:]
    assert f[:5] == [pytest.approx(100.0 ** (-j / 5), rel=1e-15) for j in range(5)]


def test_scaled_contexts():
    plain, linear = freqs(32), freqs(32, factor=8.0)
    assert linear == [pytest.approx(x / 8, rel=1e-15) for x in plain]
    parts = freqs(32, factor=8.0, original=2048.0)
    for x, y in zip(plain, parts):
        turns = 2048 * x / (2 * math.pi)
        if turns >= 32:
            assert y == pytest.approx(x, rel=1e-15)
        elif turns <= 1:
            assert y == pytest.approx(x / 8, rel=1e-15)
        else:
            assert x / 8 < y < x
    assert parts == sorted(parts, reverse=True)


@pytest.mark.parametrize("a", [(0,), (8, 3), (8, 0), (8, 9), (4097,)])
def test_refusals(a):
    with pytest.raises(sp.SpconvError):
        freqs(*a)


@pytest.mark.parametrize("k", [dict(base=1.0), dict(base=float("inf")), dict(factor=0.5), dict(original=-1.0),
                               dict(factor=float("nan"))])
def test_refused_values(k):
    with pytest.raises(sp.SpconvError):
        freqs(8, **k)
