"""A conditioned voxel block trained for a few steps: every sample of a batch of
voxel grids attends to its own states (a caption's, an image's), of any number.

    x -> layer norm -> sparse conv 3^3 -> + cross attention to the states -> z

Between the passes the block keeps its input in 8 bits only (the norm's pass
writes them), and computes the normed features again from those when the
convolution's weight gradient needs them.  The answer that is trained is one
readout per sample: a learned query that attends to the sample's voxels.

    python examples/voxel_block.py [--voxels 40000] [--channels 64] [--steps 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_convolution_gb300 as fvx  # noqa: E402
from sparse_convolution_gb300 import synth  # noqa: E402


class VoxelBlock:
    """Weights of the block and its two passes, in x's type; `group` channels
    share a step of the 8-bit input."""

    def __init__(self, channels, heads, states, samples, dtype, group=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, device="cuda", generator=g) * scale

        self.heads, self.group, self.dtype = heads, group, dtype
        size = channels // heads
        # fp32 master values; each pass reads them in its type
        self.params = {
            "norm_w": torch.ones(channels, device="cuda"),
            "norm_b": torch.zeros(channels, device="cuda"),
            "conv": normal(27, channels, channels, scale=(27 * channels) ** -0.5),
            "k": normal(states, heads, size),
            "v": normal(states, heads, size),
            "query": normal(samples, heads, size),
        }

    def weights(self):
        return {n: p if n.startswith("norm") else p.to(self.dtype) for n, p in self.params.items()}

    def forward(self, grid, kmap, x, state_offsets, state_mask):
        """The samples' readouts [samples, heads, size], and what the backward
        pass needs: x itself is not among it."""
        w = self.weights()
        n, c = x.shape
        voxels = grid.batch_offsets()
        h, mean, rstd, held = fvx.layer_norm(x, w["norm_w"], w["norm_b"], checkpoint_group=self.group)
        y = fvx.sparse_conv(grid, grid, kmap, h, w["conv"], out_dtype=self.dtype).view(n, self.heads, c // self.heads)
        seen, lse = fvx.cross_attention(y, w["k"], w["v"], voxels, state_offsets, state_mask)
        z = y + seen
        one_each = list(range(len(voxels)))
        readout, read_lse = fvx.cross_attention(w["query"], z, z, one_each, voxels)
        return readout, (w, voxels, mean, rstd, held, y, seen, lse, z, one_each, readout, read_lse)

    def backward(self, grid, kmap, kmap_t, state_offsets, state_mask, kept, dreadout):
        """Gradients of the weights, and of x."""
        w, voxels, mean, rstd, held, y, seen, lse, z, one_each, readout, read_lse = kept
        n, c = held.shape
        grad = {}
        grad["query"], dz_k, dz_v = fvx.cross_attention_backward(dreadout, w["query"], z, z, readout, read_lse,
                                                                 one_each, voxels)
        dz = dz_k + dz_v
        dq, grad["k"], grad["v"] = fvx.cross_attention_backward(dz, y, w["k"], w["v"], seen, lse, voxels,
                                                                state_offsets, state_mask)
        dy = (dz + dq).view(n, c)
        h = held.layer_norm(mean, rstd, w["norm_w"], w["norm_b"])  # from the 8 bits
        grad["conv"] = fvx.sparse_conv_wgrad(grid, grid, kmap, h, dy)
        dh = fvx.sparse_conv_dgrad(grid, grid, kmap_t, dy, w["conv"],
                                   out_dtype=self.dtype if self.dtype == torch.bfloat16 else None)
        dx, grad["norm_w"], grad["norm_b"] = fvx.layer_norm_backward(dh, held, mean, rstd, w["norm_w"])
        return grad, dx


def train(voxels=40000, channels=64, heads=4, state_lens=(77, 12, 0, 45), steps=5, rate=0.05, dtype=torch.bfloat16):
    """Trains the block towards fixed readouts; returns the losses of the steps."""
    rng = torch.Generator().manual_seed(1)
    samples = len(state_lens)
    box = max(4, round((voxels / samples * 4) ** (1 / 3)))
    coords = torch.randint(0, box, (voxels, 3), dtype=torch.int32, generator=rng).cuda()
    rows = [voxels * b // samples for b in range(samples + 1)]
    grid = fvx.Grid.build(coords, rows)
    kmap, kmap_t = fvx.KernelMap(grid, grid, 1), fvx.KernelMap(grid, grid, 1, transposed=True)
    state_offsets = [sum(state_lens[:b]) for b in range(samples + 1)]
    state_mask = (torch.rand(state_offsets[-1], generator=rng) < 0.9).cuda()
    x = torch.from_numpy(synth.features(2, grid.n_active, channels)).cuda().to(dtype)
    block = VoxelBlock(channels, heads, state_offsets[-1], samples, dtype)
    target = torch.randn(samples, heads, channels // heads, generator=rng).cuda()
    losses = []
    for _ in range(steps):
        readout, kept = block.forward(grid, kmap, x, state_offsets, state_mask)
        off = readout.float() - target
        losses.append(0.5 * float((off * off).sum()) / samples)
        grad, _ = block.backward(grid, kmap, kmap_t, state_offsets, state_mask, kept, (off / samples).to(dtype))
        for name, g in grad.items():
            block.params[name] -= rate * g.float()
    fvx.device_status()
    held = kept[4]
    print(f"{grid.n_active} voxels of {samples} samples, {channels} channels: x held in {held.nbytes} bytes, "
          f"{x.numel() * x.element_size()} in {str(dtype).split('.')[-1]}")
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--voxels", type=int, default=40000)
    p.add_argument("--channels", type=int, default=64)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args()
    for i, loss in enumerate(train(a.voxels, a.channels, steps=a.steps)):
        print(f"step {i}: loss {loss:.4f}")
