"""A residual attention block over the voxels of one cloud, forward and backward,
from the library's operators:

    u = silu(groupnorm(x))
    q, k, v = conv(u, w_qkv)                            submanifold convolution, pairs of heads on one key
    q, k turned by the voxels' coordinates              rotary positions, three axes
    a = attention(q, k, v)                              within runs of the map's schedule order
    y = x + conv(a, w_out)

    python examples/voxel_attention.py [--workload surf256] [--run 1024] [--steps 10]

trains one block on random targets and prints the loss and the time of a step.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import submanifold_sparse_convolution_spconv_amd as sp   # noqa: E402


class VoxelAttention:
    """The block's weights; convolutions in ``dtype``, the norm's in float32.
    ``heads`` heads of D = C / heads elements, of which as many pairs turn as
    divide over the three axes, on half as many heads of keys and values (2 C
    channels in all, which the convolution's gradient has kernels for)."""

    def __init__(self, C, heads, groups, K=27, dtype=torch.bfloat16, device="cuda", seed=0, causal=False):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).to(dtype).to(device)

        self.heads, self.groups, self.causal = heads, groups, causal
        self.freqs = sp.spconv_rotary_freqs(C // heads // 2 // 3 * 3, axes=3, base=100.0, device=device)
        self.params = {
            "norm_w": torch.ones(C, device=device),
            "norm_b": torch.zeros(C, device=device),
            "w_qkv": normal(K, C, 2 * C, scale=(K * C) ** -0.5),
            "w_out": normal(K, C, C, scale=(K * C) ** -0.5),
        }

    def parts(self, qkv):
        return qkv.split([self.heads, self.heads // 2, self.heads // 2], 1)

    def forward(self, x, nmap, coords, scene, order, runs):
        """x (N, C) and coords (N, 3) in the cloud's row order; scene int32 (2,),
        the rows of the cloud; order and runs: the schedule and the offsets of its
        runs.  Returns y and what the backward needs."""
        p, H = self.params, self.heads
        N, C = x.shape
        u, mean, rstd = sp.spconv_groupnorm(x, scene, self.groups, p["norm_w"], p["norm_b"], act="silu", stats=True)
        qkv = sp.spconv_forward(u, nmap, p["w_qkv"]).view(N, 2 * H, C // H)
        turned = qkv[:, :H + H // 2]
        sp.spconv_rotary(turned, coords, self.freqs, out=turned)
        q, k, v = self.parts(qkv)
        a, lse = sp.spconv_attention(q, k, v, runs, order=order, causal=self.causal, stats=True)
        y = x + sp.spconv_forward(a.view(N, C), nmap, p["w_out"])
        return y, (x, u, mean, rstd, qkv, a, lse)

    def backward(self, dy, saved, nmap, coords, scene, order, runs):
        """Returns the gradient at x and those of the weights, by name."""
        p, H = self.params, self.heads
        x, u, mean, rstd, qkv, a, lse = saved
        N, C = x.shape
        g = {"w_out": sp.spconv_wgrad(a.view(N, C), dy, nmap)}
        da = sp.spconv_dgrad(dy, nmap, p["w_out"]).view(N, H, C // H)
        dqkv = torch.empty_like(qkv)
        sp.spconv_attention_grad(da, *self.parts(qkv), a, lse, runs, order=order, causal=self.causal,
                                 grads=self.parts(dqkv))
        turned = dqkv[:, :H + H // 2]
        sp.spconv_rotary_grad(turned, coords, self.freqs, out=turned)
        dqkv = dqkv.view(N, 2 * C)
        g["w_qkv"] = sp.spconv_wgrad(u, dqkv, nmap)
        du = sp.spconv_dgrad(dqkv, nmap, p["w_qkv"])
        dx, g["norm_w"], g["norm_b"] = sp.spconv_groupnorm_grad(du, x, scene, self.groups, mean, rstd, p["norm_w"],
                                                                p["norm_b"], act="silu")
        return dy + dx, g


def main():
    import workloads as W

    a = argparse.ArgumentParser()
    a.add_argument("--workload", default="surf256")
    a.add_argument("--channels", type=int, default=128)
    a.add_argument("--heads", type=int, default=4)
    a.add_argument("--run", type=int, default=1024, help="voxels that attend to each other")
    a.add_argument("--steps", type=int, default=10)
    a.add_argument("--lr", type=float, default=0.0005)
    a = a.parse_args()
    wl = W.by_name(a.workload)
    coords = torch.from_numpy(W.geometry(wl)).cuda()
    N = coords.shape[0]
    nmap = sp.spconv_build_nmap(coords, 27, 1)
    _, order = nmap.export()
    scene = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    runs = torch.tensor(list(range(0, N, a.run)) + [N], dtype=torch.int32, device="cuda")
    x = torch.randn(N, a.channels, device="cuda").to(torch.bfloat16)
    target = torch.tanh(torch.roll(x.float(), 1, dims=1))
    block = VoxelAttention(a.channels, a.heads, groups=32)
    where = (nmap, coords, scene, order, runs)
    for step in range(a.steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        y, saved = block.forward(x, *where)
        diff = y.float() - target
        _, grads = block.backward((diff * (2 / diff.shape[1])).to(x.dtype), saved, *where)
        for name, g in grads.items():
            w = block.params[name]
            w.copy_(w.float() - a.lr * g.float() / N * a.channels)
        torch.cuda.synchronize()
        print(f"step {step}: loss {float(diff.square().mean()):.4f}, {(time.perf_counter() - t0) * 1e3:.2f} ms",
              flush=True)


if __name__ == "__main__":
    main()
