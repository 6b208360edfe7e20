"""The attention block's operators in a run, forward and backward, against
autograd of the same formulas in 64 bits; and each of them captured in a graph,
on other streams and side by side.

The longest sum has 27 C terms, seven operators stand in a row, and each rounds
to float32; the softmax multiplies what its scores are off by by their size (up
to 2 here): an output's norm is off by at most about 2 * 7 * 27 C 2^-24 of itself.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import submanifold_sparse_convolution_spconv_amd as sp

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
C, HEADS, GROUPS = 32, 2, 8
TOL = 2 * 7 * 27 * C * 2.0 ** -24


def example():
    spec = importlib.util.spec_from_file_location("voxel_attention",
                                                  os.path.join(ROOT, "examples", "voxel_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def conv(u, nbr, w):
    pad = torch.cat([u, u.new_zeros(1, u.shape[1])])
    return sum(pad[nbr[k]] @ w[k] for k in range(w.shape[0]))


def block64(p, x, nbr, coords, freqs, order, runs, causal):
    """The block's formulas on the host in 64 bits."""
    N, D = x.shape[0], C // HEADS
    t = x.view(N, GROUPS, C // GROUPS)
    var, mean = torch.var_mean(t, (0, 2), unbiased=False)
    u = ((t - mean[None, :, None]) / torch.sqrt(var + 1e-5)[None, :, None]).view(N, C) * p["norm_w"] + p["norm_b"]
    u = u * torch.sigmoid(u)
    qkv = conv(u, nbr, p["w_qkv"]).view(N, 2 * HEADS, D)
    half = HEADS // 2
    P = freqs.numel()
    angle = (coords.double()[:, torch.arange(P) // (P // 3)] * freqs)[:, None, :]
    qk = qkv[:, :HEADS + half]
    a, b, rest = qk[..., :P], qk[..., P:2 * P], qk[..., 2 * P:]
    qk = torch.cat([a * torch.cos(angle) - b * torch.sin(angle), b * torch.cos(angle) + a * torch.sin(angle), rest], -1)
    out = [None] * N
    for lo, hi in zip(runs[:-1].tolist(), runs[1:].tolist()):
        r = order[lo:hi].long()
        q, k, v = qk[r, :HEADS], *(t.repeat_interleave(2, 1) for t in (qk[r, HEADS:], qkv[r, HEADS + half:]))
        s = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
        if causal:
            s = s.masked_fill(torch.ones(hi - lo, hi - lo, dtype=torch.bool).triu(1), -float("inf"))
        o = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v)
        for i, row in enumerate(r.tolist()):
            out[row] = o[i].reshape(C)
    return x + conv(torch.stack(out), nbr, p["w_out"])


def close(got, want, what):
    err = float((got.double().cpu() - want).norm() / want.norm())
    assert err <= TOL, f"{what}: {err:.3g} of its norm off, {TOL:.3g} allowed"


@pytest.mark.parametrize("causal", [False, True])
def test_block_and_its_gradient(causal):
    rng = np.random.default_rng(3)
    coords = np.argwhere(rng.random((9, 9, 9)) < 0.4).astype(np.int32)
    coords = coords[rng.permutation(coords.shape[0])]
    N = coords.shape[0]
    cd = torch.from_numpy(coords).cuda()
    nm = sp.spconv_build_nmap(cd, 27, 1)
    _, order = nm.export()
    scene = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    runs = torch.tensor(list(range(0, N, 50)) + [N], dtype=torch.int32, device="cuda")
    block = example().VoxelAttention(C, HEADS, GROUPS, dtype=torch.float32, causal=causal)
    g = torch.Generator().manual_seed(4)
    x, dy = torch.randn(N, C, generator=g), torch.randn(N, C, generator=g)
    block.params["norm_w"] += 0.2 * torch.randn(C, generator=g).cuda()
    block.params["norm_b"] += 0.2 * torch.randn(C, generator=g).cuda()
    where = (nm, cd, scene, order, runs)
    y, saved = block.forward(x.cuda(), *where)
    dx, grads = block.backward(dy.cuda(), saved, *where)

    p = {k: v.double().cpu().requires_grad_() for k, v in block.params.items()}
    x64 = x.double().requires_grad_()
    nbr = torch.from_numpy(oracle.nmap(coords, 27, 1)).long()
    want = block64(p, x64, nbr, torch.from_numpy(coords), block.freqs.cpu(), order.cpu(), runs.cpu(), causal)
    want.backward(dy.double())
    close(y, want.detach(), "y")
    close(dx, x64.grad, "dx")
    for name, v in p.items():
        close(grads[name], v.grad, name)


def make_calls(N, dt):
    """Inputs and the operators' calls on them: small, split and shared forms."""
    H, HK, D, B = 4, 2, 40, 4
    g = torch.Generator().manual_seed(N)
    off = torch.tensor([0, N // 3, N // 3, N - 1, N], dtype=torch.int32).cuda()
    one = torch.arange(B + 1, dtype=torch.int32).cuda()
    order = torch.randperm(N, generator=g).to(torch.int32).cuda()
    pos = torch.randint(0, 1000, (N, 3), generator=g).to(torch.int32).cuda()
    freqs = sp.spconv_rotary_freqs(18, 3)
    w, b = torch.rand(H * D, generator=g).cuda(), torch.randn(H * D, generator=g).cuda()

    def inputs(seed):
        r = torch.Generator().manual_seed(seed)
        t = lambda *s: torch.randn(*s, generator=r).to(dt).cuda()
        return [t(N, H, D), t(N, HK, D), t(N, HK, D), t(N, H, D), t(B, H, D)]

    def calls(q, k, v, d, one_q):
        out, lse = sp.spconv_attention(q, k, v, off, order=order, causal=True, stats=True)
        r = [out, lse, *sp.spconv_attention_grad(d, q, k, v, out, lse, off, order=order, causal=True)]
        r += sp.spconv_attention(one_q, k, v, one, koffsets=off, korder=order, causal=True, stats=True)
        r += [sp.spconv_rotary(q, pos, freqs, gain=1.1), sp.spconv_rotary_grad(d, pos, freqs, layout="interleaved")]
        x, dx = q.view(N, H * D), d.view(N, H * D)
        y, mean, rstd = sp.spconv_groupnorm(x, off, 8, w, b, act="gelu", stats=True)
        return r + [y, mean, rstd, *sp.spconv_groupnorm_grad(dx, x, off, 8, mean, rstd, w, b, act="gelu")]

    return inputs, calls


@pytest.mark.parametrize("N, dt", [(37, torch.float32), (1500, torch.bfloat16), (20000, torch.bfloat16)])
def test_operators_in_a_graph(N, dt):
    """Captured once, replayed on new inputs with eager work between: the bits of
    the eager calls."""
    inputs, calls = make_calls(N, dt)
    held = inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(*held)
    for seed in range(1, 5):
        new = inputs(seed)
        want = calls(*new)
        for a, b in zip(held, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"output {i}"


def test_two_streams_at_once():
    """Calls of two streams that overlap do not share anything."""
    inputs, calls = make_calls(6000, torch.bfloat16)
    one, two = inputs(1), inputs(2)
    want = [calls(*one), calls(*two)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, t in enumerate((one, two)):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls(*t))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)


def test_callers_workspaces():
    """The caller's workspace, whatever it holds, and none that is too small."""
    q = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(30000, 2, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    o, ko = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (1, 30000))
    n = sp.spconv_attention_workspace_size(1, 30000, 1, 8, 2, 128, sp.SPCONV_BF16)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    want = sp.spconv_attention(q, k, v, o, koffsets=ko)
    assert torch.equal(sp.spconv_attention(q, k, v, o, koffsets=ko, workspace=ws), want)
    with pytest.raises(ValueError):
        sp.spconv_attention(q, k, v, o, koffsets=ko, workspace=ws[:-1])
    x = torch.randn(3000, 64, device="cuda")
    off = torch.tensor([0, 1000, 3000], dtype=torch.int32, device="cuda")
    n = sp.spconv_groupnorm_workspace_size(3000, 64, 2, 4, sp.SPCONV_F32)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(sp.spconv_groupnorm(x, off, 4, workspace=ws), sp.spconv_groupnorm(x, off, 4))


def test_refusals_on_the_card():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    o = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    q, k = t(8, 4, 32), t(8, 2, 32)
    bad = [
        lambda: sp.spconv_attention(q, k, t(8, 2, 32, dt=torch.float32), o),
        lambda: sp.spconv_attention(q, k, t(7, 2, 32), o),
        lambda: sp.spconv_attention(q, t(8, 3, 32), t(8, 3, 32), o),
        lambda: sp.spconv_attention(q, t(9, 2, 32), t(9, 2, 32), o),
        lambda: sp.spconv_attention(q, k, k, o.long()),
        lambda: sp.spconv_attention(q, k, k, o, korder=o),
        lambda: sp.spconv_attention(q, k, k, o, koffsets=torch.zeros(3, dtype=torch.int32, device="cuda")),
        lambda: sp.spconv_attention(q, k, k, o, order=o),
        lambda: sp.spconv_attention(q, k, k, o, out=t(8, 4, 33)[..., :32]),
        lambda: sp.spconv_attention(t(8, 4, 32, dt=torch.float16), k, k, o),
        lambda: sp.spconv_groupnorm(t(8, 32), o, 4, weight=t(32)),
        lambda: sp.spconv_groupnorm(t(8, 32), o, 4, act="relu"),
        lambda: sp.spconv_rotary(q, o, torch.ones(4, device="cuda")),
        lambda: sp.spconv_rotary(q, o[:1].expand(8), torch.ones(4, device="cuda", dtype=torch.float64), layout="x"),
        lambda: sp.spconv_rotary(q, o, torch.ones(4, device="cuda", dtype=torch.float64)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(str(i))
    for f in (lambda: sp.spconv_groupnorm(t(8, 32), o, 5), lambda: sp.spconv_attention(q, k, k, o, scale=0.0),
              lambda: sp.spconv_attention(t(8, 4, 20), t(8, 2, 20), t(8, 2, 20), o),
              lambda: sp.spconv_attention(t(8 * 4 * 32 + 1)[1:].view(8, 4, 32), k, k, o)):
        with pytest.raises(sp.SpconvError):
            f()
