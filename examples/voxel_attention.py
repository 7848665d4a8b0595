"""Voxels that attend to the voxels of their own sample, trained for a few steps:
the positions are their coordinates.

    x -> layer norm -> queries, keys, values -> norms per head and rotation by
    (i, j, k) -> attention -> product -> dropout, added to x -> y

Queries and keys are normed and turned out of one product's rows in one pass, and
their gradients written back into one such tensor.  No mask of the dropout is
kept: the backward pass draws it again.

    python examples/voxel_attention.py [--voxels 8000] [--channels 128] [--steps 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_convolution_gb300 as fvx  # noqa: E402


class VoxelAttention:
    """Weights of the block and its two passes, in x's type; call `step` numbers
    the dropout's draws."""

    def __init__(self, channels, heads, dtype, p=0.1, base=100.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, device="cuda", generator=g) * shape[0] ** -0.5

        self.heads, self.size, self.dtype, self.p, self.seed = heads, channels // heads, dtype, p, seed
        self.rotary = fvx.Rotary(self.size // 2 * 2, axes=3, base=base)
        # fp32 master values; each pass reads the matrices in its type
        self.params = {
            "norm_w": torch.ones(channels, device="cuda"),
            "norm_b": torch.zeros(channels, device="cuda"),
            "qkv": normal(channels, 3 * channels),
            "q_w": torch.ones(self.size, device="cuda"),
            "k_w": torch.ones(self.size, device="cuda"),
            "out": normal(channels, channels),
        }

    def weights(self):
        return {n: p.to(self.dtype) if p.dim() == 2 else p for n, p in self.params.items()}

    def forward(self, grid, x, step):
        """y [voxels, channels], and what the backward pass needs."""
        w, h, n = self.weights(), self.heads, x.shape[0]
        voxels, ijk = grid.batch_offsets(), grid.ijk()
        normed, mean, rstd = fvx.layer_norm(x, w["norm_w"], w["norm_b"])
        qkv = (normed @ w["qkv"]).view(n, 3 * h, self.size)
        q, k = fvx.norm_rotate_heads(qkv[:, :h], ijk, self.rotary, w["q_w"], k=qkv[:, h:2 * h], k_weight=w["k_w"])
        seen, lse = fvx.cross_attention(q, k, qkv[:, 2 * h:], voxels, voxels)
        y = fvx.dropout(seen.view(n, -1) @ w["out"], self.p, self.seed, step, residual=x)
        return y, (w, voxels, ijk, step, x, normed, mean, rstd, qkv, q, k, seen, lse)

    def backward(self, kept, dy):
        """Gradients of the weights, and of x."""
        w, voxels, ijk, step, x, normed, mean, rstd, qkv, q, k, seen, lse = kept
        h, n = self.heads, x.shape[0]
        grad = {}
        do = fvx.dropout_backward(dy, self.p, self.seed, step)
        grad["out"] = seen.view(n, -1).t() @ do
        dseen = (do @ w["out"].t()).view_as(seen)
        dq, dk, dv = fvx.cross_attention_backward(dseen, q, k, qkv[:, 2 * h:], seen, lse, voxels, voxels)
        dqkv = torch.empty_like(qkv)
        _, _, grad["q_w"], grad["k_w"] = fvx.norm_rotate_heads_backward(
            dq, qkv[:, :h], ijk, self.rotary, w["q_w"], dk=dk, k=qkv[:, h:2 * h], k_weight=w["k_w"],
            out=(dqkv[:, :h], dqkv[:, h:2 * h]))
        dqkv[:, 2 * h:] = dv
        dqkv = dqkv.view(n, -1)
        grad["qkv"] = normed.t() @ dqkv
        dx, grad["norm_w"], grad["norm_b"] = fvx.layer_norm_backward(dqkv @ w["qkv"].t(), x, mean, rstd, w["norm_w"])
        return grad, dy + dx


def train(voxels=8000, channels=128, heads=4, samples=3, steps=5, rate=0.02, dtype=torch.bfloat16):
    """Trains the block towards a fixed shift of its input; returns the steps' losses."""
    rng = torch.Generator().manual_seed(1)
    box = max(4, round((voxels / samples * 4) ** (1 / 3)))
    coords = torch.randint(0, box, (voxels, 3), dtype=torch.int32, generator=rng).cuda()
    grid = fvx.Grid.build(coords, [voxels * b // samples for b in range(samples + 1)])
    x = torch.randn(grid.n_active, channels, generator=rng).cuda().to(dtype)
    target = x.float() + torch.randn(channels, generator=rng).cuda()
    block = VoxelAttention(channels, heads, dtype)
    losses = []
    for step in range(steps):
        y, kept = block.forward(grid, x, step)
        off = y.float() - target
        losses.append(0.5 * float((off * off).mean()))
        grad, _ = block.backward(kept, (off / off.shape[0]).to(dtype))
        for name, g in grad.items():
            block.params[name] -= rate * g.float()
    fvx.device_status()
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--voxels", type=int, default=8000)
    p.add_argument("--channels", type=int, default=128)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args()
    for i, loss in enumerate(train(a.voxels, a.channels, steps=a.steps)):
        print(f"step {i}: loss {loss:.4f}")
