"""The gradient's weights exp(score - lse) of a query sum to one.  Scores are
multiplied by scale log2 e, rounded to 32 bits; lse has to follow that rounding, or
all weights are off the same way, by the score times the rounding (2^-25 to 2^-24).

Seen in sum_j dv[j] = sum_i (sum_j p[i, j]) dout[i], 1 for each query where dout is
1: the mean over n queries whose lse is about L = 90.  What a query's sum is off by at
random, half a step of lse (2^-18 at 90) and of lse log2 e (2^-17) and a step of
every weight's exponent (2^-17 ln 2, the same size), has a root mean square below
2^-17 and a mean over n = 4,096 queries below 6 2^-17 / 64 = 7.2e-7 (six sigma).  What
remains of the rounding of scale, 2^-24 of log sum exp(score - largest) <= 6, adds
3.6e-7.  Going by log2 e it would be 85 times the rounding, 2^-24.4 and 2^-23.7 of
the scales chosen here: 3.9e-6 and 6.1e-6.
"""
import math
import struct

import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp
from kernel_names import assert_launches

pytestmark = pytest.mark.gpu


def f32(x):
    return struct.unpack("f", struct.pack("f", x))[0]


def rounding(scale):
    """Of scale log2 e in 32 bits, relative."""
    exact = scale * math.log2(math.e)
    return f32(f32(scale) * f32(math.log2(math.e))) / exact - 1


# scales about 0.35 whose product is rounded far up, and far down
SCALES = [pick((f32(0.35 + i * 2.0 ** -24) for i in range(4000)), key=rounding) for pick in (max, min)]


@pytest.mark.parametrize("L, B, kernel", [(256, 16, 0), (64, 64, 0), (8, 512, 1)])
@pytest.mark.parametrize("scale", SCALES, ids=["up", "down"])
def test_weights_sum_to_one(L, B, kernel, scale):
    assert abs(rounding(scale)) > 2.0 ** -24.5
    N, H, D = L * B, 4, 8
    g = torch.Generator().manual_seed(L)
    q, k = (torch.randn(N, H, D, generator=g) * 0.5 for _ in range(2))
    q[..., 0] = k[..., 0] = (85 / scale) ** 0.5
    v, do = torch.randn(N, H, D, generator=g), torch.ones(N, H, D)
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    o = torch.arange(0, N + 1, L, dtype=torch.int32, device="cuda")
    out, lse = sp.spconv_attention(q, k, v, o, scale=scale, stats=True)
    assert 80 < float(lse.min()) and float(lse.max()) < 100
    grad = lambda: sp.spconv_attention_grad(do, q, k, v, out, lse, o, scale=scale)
    assert_launches(grad, f"k_attn_dkv<f32, 32, {kernel}>")
    sums = grad()[2].double().sum((0, 2)) / (N * D)
    print([float(s) for s in sums - 1])
    assert float((sums - 1).abs().max()) <= 6 * 2.0 ** -17 / 64 + 6 * 2.0 ** -24
