"""Sizes of the row operators at the edge of what a launch can hold (no GPU
needed: only sizes are asked for)."""
import ctypes

import submanifold_sparse_convolution_spconv_amd as sp

OK, UNSUPPORTED = 0, -2


def test_scan_of_more_threads_than_a_launch_has():
    """64 rows of 65 channels take a workgroup of 512: 2^23 of them are 2^32
    threads (the gradient); the forward's take twice the rows."""
    lib = sp.load_library()
    n = ctypes.c_size_t(0)
    grad = lambda N, C: lib.spconv_scan_grad_workspace_size(N, C, 1, ctypes.byref(n))
    fwd = lambda N, C: lib.spconv_scan_workspace_size(N, C, 1, ctypes.byref(n))
    assert grad((1 << 29) - 64, 65) == OK
    assert grad((1 << 29) - 63, 65) == UNSUPPORTED and b"2^32 threads" in lib.spconv_last_error()
    assert fwd((1 << 30) - 128, 65) == OK and fwd((1 << 30) - 127, 65) == UNSUPPORTED
    # two tiles of channels, whose chunks go round eight XCDs
    assert grad((1 << 28) - 64 * 8, 129) == OK and grad(1 << 28, 129) == UNSUPPORTED
    assert grad((1 << 31) - 2, 4) == OK and fwd((1 << 31) - 2, 16) == OK


def test_refused_scans_enqueue_nothing():
    lib = sp.load_library()
    p = ctypes.c_void_p(0x7f0000000000)          # aligned, never dereferenced
    N = (1 << 29) + 64
    assert lib.spconv_scan_grad(p, p, p, p, None, None, None, p, 1 << 40, p, p, None, N, 65, 1, 1, None) == UNSUPPORTED
    assert lib.spconv_scan(p, p, p, None, None, p, 1 << 40, p, p, 2 * N, 65, 1, 1, None) == UNSUPPORTED
