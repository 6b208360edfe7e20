"""The ends of the operators' ranges within scenes (no GPU needed): sizes that a
kernel's 32-bit counts of rows cannot hold are refused, and the largest ones that
they can are not."""
import ctypes

import pytest

import submanifold_sparse_convolution_spconv_amd as sp

OK, UNSUPPORTED, WORKSPACE = 0, -2, -5
LAST = (1 << 31) - 1024         # rows of a sequence: the loops look up to 8 tiles of 64 rows past the end


@pytest.fixture(scope="module")
def lib():
    return sp.load_library()


def test_attention_rows_past_31_bits(lib):
    """Tiles past the last row are numbered too (tile * rows + row): their numbers
    have to stay within 31 bits, for keys, and for queries times the heads that
    share keys."""
    n = ctypes.c_size_t(0)
    for S in (lib.spconv_attention_workspace_size, lib.spconv_attention_grad_workspace_size):
        Z = lambda N, M, G=1: S(N, M, 1, G, 1, 8, sp.SPCONV_BF16, ctypes.byref(n))
        for past in (LAST + 1, (1 << 31) - 256, (1 << 31) - 128, (1 << 31) - 64, (1 << 31) - 2, (1 << 31) - 1):
            assert Z(1, past) == UNSUPPORTED and Z(past, 1) == UNSUPPORTED, past
        assert Z(LAST // 8 + 1, 1, G=8) == UNSUPPORTED and Z((1 << 28) - 1, 1, G=8) == UNSUPPORTED
    assert lib.spconv_attention_workspace_size(1, LAST, 1, 1, 1, 8, sp.SPCONV_BF16, ctypes.byref(n)) == OK


def test_attention_threads_are_counted_by_the_kernel_taken(lib):
    """A launch's threads are counted in 32 bits.  Calls of many rows have 128 of them
    a workgroup: 11 million rows (the largest cloud here) of 32 heads are an eighth of
    the limit, not past it."""
    n = ctypes.c_size_t(0)
    for S in (lib.spconv_attention_workspace_size, lib.spconv_attention_grad_workspace_size):
        Z = lambda N, B, H=32: S(N, N, B, H, H, 8, sp.SPCONV_BF16, ctypes.byref(n))
        assert Z(11_000_000, 11_000) == OK
        # (N / 128 + B) 32 workgroups of 256 threads, in runs of 64
        assert Z((1 << 26) - (1 << 14), 1) == OK and Z((1 << 26) - 128, 1) == UNSUPPORTED
        # sequences of few rows: 16 or 32 rows a workgroup, and one for each sequence at least
        assert Z(1 << 19, 1 << 19, H=16) == OK and Z(1 << 20, 1 << 20, H=16) == UNSUPPORTED
        assert Z(1, (1 << 24) - 128, H=1) == OK and Z(1, 1 << 24, H=1) == UNSUPPORTED


def test_groupnorm_gradient_counts_its_channel_sums(lib):
    """The gradient's launch that joins scenes and groups has workgroups for dweight
    and dbias too: with them 2^32 threads are reached where the forward's are not."""
    p = ctypes.c_void_p(0x7f0000000000)         # never read: every call fails a check
    n = ctypes.c_size_t(0)
    C, G = 4096, 4
    for B, want in (((1 << 20) - 1, UNSUPPORTED), ((1 << 20) - 100, UNSUPPORTED), ((1 << 20) - 128 - 1, WORKSPACE)):
        assert lib.spconv_groupnorm_workspace_size(1, C, B, G, sp.SPCONV_BF16, ctypes.byref(n)) == OK
        assert lib.spconv_groupnorm(p, p, None, None, p, 0, p, None, None, 1, C, B, G, 1e-5, 0, sp.SPCONV_BF16,
                                    None) == WORKSPACE
        assert lib.spconv_groupnorm_grad(p, p, p, p, p, None, None, p, 0, p, p, p, 1, C, B, G, 0, sp.SPCONV_BF16,
                                         None) == want, B
