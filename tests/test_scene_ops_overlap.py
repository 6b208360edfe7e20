"""Outputs whose rows or heads lie in one another are refused (no GPU needed): an
expanded tensor's elements would be written by several workgroups at once."""
import ctypes

import pytest

import submanifold_sparse_convolution_spconv_amd as sp

FAKE = ctypes.c_void_p(0x7f0000000000)         # never read: every call fails a check
INVALID, WORKSPACE = -1, -5
N, H, HK, D = 64, 4, 2, 64
GOOD = (H * D, D)
# expanded rows, expanded heads, rows that begin inside others, heads that do
BAD = [(0, D), (H * D, 0), (H * D - 8, D), (D, D), (D, (N - 1) * D), (H * D, D - 8)]
FINE = [GOOD, (D, N * D), (2 * H * D, D), (3 * H * D, 2 * D)]


@pytest.fixture(scope="module")
def lib():
    return sp.load_library()


def strides(*pairs):
    flat = [n for p in pairs for n in p]
    return (ctypes.c_int64 * len(flat))(*flat)


def test_attention(lib):
    kv = (HK * D, D)

    def forward(out):
        return lib.spconv_attention(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, strides(GOOD, kv, kv, out), FAKE, 0, FAKE,
                                    None, N, 100000, 1, H, HK, D, 0.1, 0, sp.SPCONV_BF16, None)

    def gradient(dq=GOOD, dk=kv, dv=kv, out=GOOD):
        return lib.spconv_attention_grad(*[FAKE] * 7, None, None, None, strides(GOOD, kv, kv, out, GOOD, dq, dk, dv),
                                         FAKE, 0, FAKE, FAKE, FAKE, N, N, 1, H, HK, D, 0.1, 0, sp.SPCONV_BF16, None)
    for s in FINE:
        assert forward(s) == WORKSPACE and gradient(dq=s) == WORKSPACE, s
    for s in BAD:
        assert forward(s) == INVALID and gradient(dq=s) == INVALID, s
        assert gradient(out=s) == WORKSPACE, s                       # an input may be expanded
    for s in ((0, D), (HK * D, 0), (D, D), (HK * D - 8, D)):
        assert gradient(dk=s) == INVALID and gradient(dv=s) == INVALID, s


def test_rotary(lib):
    for s in BAD:
        for x in (FAKE.value, FAKE.value + (1 << 30)):               # in place, and not
            assert lib.spconv_rotary(ctypes.c_void_p(x), FAKE, 1, FAKE, FAKE, strides(s, s), N, H, D, 16, 1, 0, 1.0,
                                     sp.SPCONV_BF16, None) == INVALID, s
