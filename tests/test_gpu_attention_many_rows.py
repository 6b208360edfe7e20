"""Attention of more rows times heads than a launch of 16 rows a workgroup could
count: 11 million rows of 32 heads, sequences of 1,000 rows, some of them against
64 bits."""
import pytest
import torch

import submanifold_sparse_convolution_spconv_amd as sp
from attn_ref import attention64, check

pytestmark = pytest.mark.gpu


def test_eleven_million_rows():
    B, L, H, D = 11_000, 1_000, 32, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn(B * L, H, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    o = torch.arange(0, B * L + 1, L, dtype=torch.int32, device="cuda")
    print("forward", flush=True)
    out, lse = sp.spconv_attention(q, k, v, o, causal=True, stats=True)
    torch.cuda.synchronize()
    print("gradient", flush=True)
    grads = sp.spconv_attention_grad(do, q, k, v, out, lse, o, causal=True)
    torch.cuda.synchronize()
    for b in (0, 5_432, B - 1):
        # heads stand alone: two of them say enough
        part = lambda t: t[b * L:(b + 1) * L, ::31].contiguous()
        want = attention64(part(q), part(k), part(v), torch.tensor([0, L]), causal=True, dout=part(do))
        for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            check(part(t), want[name], f"{name} of sequence {b}")
