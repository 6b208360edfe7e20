"""Refusals of the operators within scenes (no GPU needed): the C entry points'
checks return the documented codes before anything is enqueued, and the Python
functions refuse tensors that do not fit."""
import ctypes

import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp

FAKE = 0x7f0000000000           # aligned, never dereferenced: every call below fails a check or has no rows
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -5


@pytest.fixture(scope="module")
def lib():
    return sp.load_library()


def p(a):
    return ctypes.c_void_p(a) if a else None


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def test_rotary_refusals(lib):
    for fn in (lib.spconv_rotary, lib.spconv_rotary_grad):
        def f(x=FAKE, pos=FAKE, fr=FAKE, y=FAKE + 4096, st=None, N=4, H=2, D=32, P=12, axes=3, lay=0, dt=1):
            return fn(p(x), p(pos), axes, p(fr), p(y), st, N, H, D, P, axes, lay, 1.0, dt, None)
        assert f(N=0) == OK and f(N=0, x=0, pos=0, fr=0, y=0) == OK
        for k in ("x", "pos", "fr", "y"):
            assert f(**{k: 0}) == INVALID, k
        assert f(x=FAKE + 1) == INVALID and f(y=FAKE + 2, dt=0) == INVALID and f(pos=FAKE + 2) == INVALID
        assert f(fr=FAKE + 4) == INVALID
        assert f(N=-1) == INVALID and f(N=1 << 31) == UNSUPPORTED
        assert f(H=0) == INVALID and f(H=4097) == UNSUPPORTED and f(D=4097) == UNSUPPORTED and f(D=0) == INVALID
        assert f(P=18) == INVALID and f(P=0) == INVALID and f(P=13) == INVALID      # beyond D, none, not by axes
        assert f(axes=0) == INVALID and f(axes=9, P=9) == INVALID
        assert f(lay=2) == INVALID and f(dt=2) == INVALID
        assert f(y=FAKE, st=strides(64, 32, 128, 32)) == INVALID                    # in place, other strides


def test_groupnorm_refusals(lib):
    n = ctypes.c_size_t(0)
    S = lambda N, C, B, G, dt: lib.spconv_groupnorm_workspace_size(N, C, B, G, dt, ctypes.byref(n))
    assert S(1006716, 128, 4, 32, 1) == OK and 0 < n.value < 8 << 20 and n.value % 256 == 0
    assert S(10, 128, 0, 32, 1) == INVALID and S(10, 128, 4, 0, 1) == INVALID and S(10, 128, 4, 3, 1) == INVALID
    assert S(10, 4097, 4, 1, 1) == UNSUPPORTED and S(-1, 8, 1, 1, 1) == INVALID and S(1, 8, 1, 1, 5) == INVALID
    assert S(1 << 31, 8, 1, 1, 1) == UNSUPPORTED and S(1, 64, 1 << 20, 32, 1) == UNSUPPORTED
    assert lib.spconv_groupnorm_workspace_size(4, 64, 1, 8, 1, None) == INVALID
    assert S(4, 64, 3, 8, 1) == OK
    need = n.value

    def f(x=FAKE, off=FAKE, w=FAKE, b=FAKE, ws=FAKE, wb=need, y=FAKE, m=FAKE, r=FAKE, N=4, C=64, B=3, G=8, eps=1e-5,
          act=0, dt=1):
        return lib.spconv_groupnorm(p(x), p(off), p(w), p(b), p(ws), wb, p(y), p(m), p(r), N, C, B, G, eps, act, dt,
                                    None)
    for k in ("x", "off", "ws", "y", "m", "r"):
        assert f(**{k: 0}) == INVALID, k
    assert f(wb=need - 1) == WORKSPACE and f(ws=FAKE + 64) == INVALID and f(x=FAKE + 1) == INVALID
    assert f(w=FAKE + 2) == INVALID and f(m=FAKE + 2) == INVALID and f(off=FAKE + 1) == INVALID
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID and f(act=3) == INVALID and f(act=-1) == INVALID
    assert f(G=5) == INVALID and f(B=0) == INVALID and f(dt=2) == INVALID and f(C=5000, G=1) == UNSUPPORTED

    def g(d=FAKE, x=FAKE, off=FAKE, m=FAKE, r=FAKE, ws=FAKE, wb=need, dx=FAKE, dw=FAKE, db=FAKE, act=0):
        return lib.spconv_groupnorm_grad(p(d), p(x), p(off), p(m), p(r), None, None, p(ws), wb, p(dx), p(dw), p(db), 4,
                                         64, 3, 8, act, 1, None)
    for k in ("d", "x", "off", "m", "r", "ws", "dx", "dw", "db"):
        assert g(**{k: 0}) == INVALID, k
    assert g(wb=0) == WORKSPACE and g(act=9) == INVALID and g(d=FAKE + 1) == INVALID


def test_attention_refusals(lib):
    n = ctypes.c_size_t(0)
    for S in (lib.spconv_attention_workspace_size, lib.spconv_attention_grad_workspace_size):
        Z = lambda N=64, M=64, B=2, H=4, HK=2, D=64, dt=1: S(N, M, B, H, HK, D, dt, ctypes.byref(n))
        assert Z() == OK and n.value % 256 == 0
        assert Z(N=1006716, M=1006716, B=984, D=32) == OK and n.value <= 1006716 * 4 * 4 + 256
        assert Z(D=0) == INVALID and Z(D=12) == UNSUPPORTED and Z(D=136) == UNSUPPORTED
        assert Z(H=3) == INVALID and Z(HK=0) == INVALID and Z(H=8192) == UNSUPPORTED and Z(B=0) == INVALID
        assert Z(N=-1) == INVALID and Z(M=-1) == INVALID and Z(N=1 << 31) == UNSUPPORTED and Z(dt=3) == INVALID
        assert Z(N=1 << 30, H=4, HK=1) == UNSUPPORTED and Z(B=(1 << 31) - 1) == UNSUPPORTED
        assert S(1, 1, 1, 1, 1, 8, 1, None) == INVALID
    assert lib.spconv_attention_workspace_size(1, 100000, 1, 8, 2, 128, 1, ctypes.byref(n)) == OK and n.value > 0
    split = n.value

    def f(q=FAKE, k=FAKE, v=FAKE, off=FAKE, ko=None, o=None, ko2=None, st=None, ws=None, wb=0, out=FAKE, lse=FAKE, N=64,
          M=64, B=2, H=4, HK=2, D=64, scale=0.1, dt=1):
        return lib.spconv_attention(p(q), p(k), p(v), p(off), p(ko), p(o), p(ko2), st, p(ws), wb, p(out), p(lse), N, M,
                                    B, H, HK, D, scale, 0, dt, None)
    assert f(N=0, M=0, q=0, k=0, v=0, out=0) == OK                  # nothing to do
    for k in ("q", "k", "v", "off", "out"):
        assert f(**{k: 0}) == INVALID, k
    for k in ("q", "k", "v", "out"):
        assert f(**{k: FAKE + 8}) == INVALID, k
    assert f(M=65) == INVALID and f(ko2=FAKE) == INVALID            # other keys need their offsets
    assert f(off=FAKE + 2) == INVALID and f(lse=FAKE + 1) == INVALID and f(o=FAKE + 2) == INVALID
    assert f(scale=0.0) == INVALID and f(scale=-1.0) == INVALID and f(scale=float("inf")) == INVALID
    assert f(scale=float("nan")) == INVALID and f(dt=2) == INVALID and f(D=20) == UNSUPPORTED
    good = [256, 64, 128, 64, 128, 64, 256, 64]
    for i in range(8):
        bad = list(good)
        bad[i] += 4
        assert f(st=strides(*bad)) == INVALID, i
        bad[i] = -8
        assert f(st=strides(*bad)) == INVALID, i
    assert f(st=strides(256, 64, (1 << 23) + 8, 64, 128, 64, 256, 64)) == UNSUPPORTED      # rows too far apart
    long = dict(N=1, M=100000, B=1, H=8, D=128, ko=FAKE)
    assert f(**long) == INVALID and f(**long, ws=FAKE, wb=split - 1) == WORKSPACE
    assert f(**long, ws=FAKE + 128, wb=split) == INVALID
    assert lib.spconv_attention_grad_workspace_size(64, 64, 2, 4, 2, 64, 1, ctypes.byref(n)) == OK
    need = n.value

    def g(d=FAKE, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, off=FAKE, st=None, ws=FAKE, wb=need, dq=FAKE, dk=FAKE,
          dv=FAKE, scale=0.1):
        return lib.spconv_attention_grad(p(d), p(q), p(k), p(v), p(out), p(lse), p(off), None, None, None, st, p(ws), wb,
                                         p(dq), p(dk), p(dv), 64, 64, 2, 4, 2, 64, scale, 1, 1, None)
    for k in ("d", "q", "k", "v", "out", "lse", "off", "ws", "dq", "dk", "dv"):
        assert g(**{k: 0}) == INVALID, k
    for k in ("d", "out", "dq", "dk", "dv"):
        assert g(**{k: FAKE + 8}) == INVALID, k
    assert g(wb=need - 1) == WORKSPACE and g(scale=0.0) == INVALID
    assert g(st=strides(*(good + [256, 64, 256, 64, 128, 64, 128, 65]))) == INVALID


def test_python_refuses_host_tensors():
    x, h = torch.zeros(4, 64), torch.zeros(4, 2, 32)
    o = torch.tensor([0, 4], dtype=torch.int32)
    for call in (lambda: sp.spconv_groupnorm(x, o, 8), lambda: sp.spconv_groupnorm_grad(x, x, o, 8, x, x),
                 lambda: sp.spconv_rotary(h, o[:1].expand(4), torch.ones(4, dtype=torch.float64)),
                 lambda: sp.spconv_rotary_grad(h, o, None), lambda: sp.spconv_attention(h, h, h, o),
                 lambda: sp.spconv_attention_grad(h, h, h, h, h, h[..., 0], o), lambda: sp.spconv_attention(h, h, None, o)):
        with pytest.raises(ValueError):
            call()
