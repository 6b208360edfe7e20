"""A residual block over the voxels of one cloud, forward and backward, from the
library's operators:

    u = layernorm(x)
    v = conv(u, w_value),  z = conv(u, w_gate)          submanifold convolutions
    h = scan(v, z)                                      along the map's schedule order
    y = x + glu(h)

    python examples/voxel_block.py [--workload surf256] [--steps 10]

trains one block on random targets and prints the loss and the time of a step.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import submanifold_sparse_convolution_spconv_amd as sp   # noqa: E402


class VoxelBlock:
    """The block's weights; convolutions and the gated unit in ``dtype``, the
    norm's and the biases in float32."""

    def __init__(self, C, K=27, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale, dt=dtype):
            return (torch.randn(*shape, generator=g) * scale).to(dt).to(device)

        self.params = {
            "norm_w": torch.ones(C, device=device),
            "norm_b": torch.zeros(C, device=device),
            "w_value": normal(K, C, C, scale=(K * C) ** -0.5),
            "w_gate": normal(K, C, C, scale=(K * C) ** -0.5),
            "w_glu": normal(2, C, C, scale=C ** -0.5),
            "b_glu": torch.zeros(2, C, device=device),
        }

    def forward(self, x, nmap, order, offsets):
        """x (N, C) in the cloud's row order.  Returns y and what the backward
        needs."""
        p = self.params
        u, mean, rstd = sp.spconv_layernorm(x, p["norm_w"], p["norm_b"], stats=True)
        v = sp.spconv_forward(u, nmap, p["w_value"])
        z = sp.spconv_forward(u, nmap, p["w_gate"])
        h, _ = sp.spconv_scan(v, z, offsets, order=order)
        y = x + sp.spconv_glu(h, p["w_glu"], p["b_glu"])
        return y, (x, u, mean, rstd, v, z, h)

    def backward(self, dy, saved, nmap, order, offsets):
        """Returns the gradient at x and those of the weights, by name."""
        p = self.params
        x, u, mean, rstd, v, z, h = saved
        g = {}
        dh, g["w_glu"], g["b_glu"] = sp.spconv_glu_grad(dy, h, p["w_glu"], p["b_glu"])
        dv, dz, _ = sp.spconv_scan_grad(dh, v, z, offsets, order=order)
        g["w_value"] = sp.spconv_wgrad(u, dv, nmap)
        g["w_gate"] = sp.spconv_wgrad(u, dz, nmap)
        du = sp.spconv_dgrad(dv, nmap, p["w_value"]) + sp.spconv_dgrad(dz, nmap, p["w_gate"])
        dx, g["norm_w"], g["norm_b"] = sp.spconv_layernorm_grad(du, x, mean, rstd, p["norm_w"])
        return dy + dx, g


def main():
    import workloads as W

    a = argparse.ArgumentParser()
    a.add_argument("--workload", default="surf256")
    a.add_argument("--channels", type=int, default=128)
    a.add_argument("--steps", type=int, default=10)
    a.add_argument("--lr", type=float, default=0.05)
    a = a.parse_args()
    wl = W.by_name(a.workload)
    coords = torch.from_numpy(W.geometry(wl)).cuda()
    N = coords.shape[0]
    nmap = sp.spconv_build_nmap(coords, 27, 1)
    _, order = nmap.export()
    offsets = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    x = torch.randn(N, a.channels, device="cuda").to(torch.bfloat16)
    target = torch.tanh(torch.roll(x.float(), 1, dims=1))
    block = VoxelBlock(a.channels)
    for step in range(a.steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        y, saved = block.forward(x, nmap, order, offsets)
        diff = y.float() - target
        _, grads = block.backward((diff * (2 / diff.shape[1])).to(x.dtype), saved, nmap, order, offsets)
        for name, g in grads.items():
            w = block.params[name]
            w.copy_(w.float() - a.lr * g.float() / N * a.channels)
        torch.cuda.synchronize()
        print(f"step {step}: loss {float(diff.square().mean()):.4f}, {(time.perf_counter() - t0) * 1e3:.2f} ms",
              flush=True)


if __name__ == "__main__":
    main()
