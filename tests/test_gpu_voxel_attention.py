"""The example that runs head norms, rotation, attention and dropout together
(examples/voxel_attention.py): its output and gradients against the formulas in
64 bits, and its passes as often as they are asked for."""
from __future__ import annotations

import numpy as np
import pytest

from tests.helpers_dropout import kept as drawn

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _grid(voxels, samples, box, seed):
    import sparse_convolution_gb300 as fvx

    g = torch.Generator().manual_seed(seed)
    coords = torch.randint(-box // 2, box, (voxels, 3), dtype=torch.int32, generator=g).cuda()
    grid = fvx.Grid.build(coords, [voxels * b // samples for b in range(samples + 1)])
    return grid, g


def _angles(rotary, ijk):
    """[voxels, pairs] radians, exactly from the steps' integers."""
    pairs = rotary.size // 2
    axis = np.repeat(np.arange(3), [pairs // 3 + (a < pairs % 3) for a in range(3)])
    at = ijk.cpu().numpy().astype(np.int64)[:, axis].astype(np.uint64)
    with np.errstate(over="ignore"):
        part = (at * rotary.turns[None]).astype(np.int64)
    return torch.from_numpy(part.astype(np.float64) / 2.0 ** 64 * (2 * np.pi))


def test_gradients_match_the_formulas():
    """fp32 against autograd in 64 bits.

    Tolerance, of the largest value of each tensor: an fp32 sum of n terms
    wanders from the exact one by about sqrt(n) 2^-24 of its terms' root sum of
    squares; the longest sums here have 1200 terms (over the voxels), so about 35
    * 6e-8 = 2.1e-6 per operator, and the chain has seven of them, forward and
    back.  Scores of normed heads of 24 values reach sqrt(24) = 5, which their
    errors multiply by; differences (softmax's and the norms' gradients) lose up
    to a factor of about 10 where they nearly cancel: 7 * 5 * 10 * 2.1e-6 =
    7e-4, taken as 8e-4."""
    import sparse_convolution_gb300 as fvx
    from examples.voxel_attention import VoxelAttention

    grid, g = _grid(1200, 3, 14, 3)
    n, channels, heads = grid.n_active, 72, 3
    block = VoxelAttention(channels, heads, torch.float32, p=0.2)
    for name in ("norm_w", "q_w", "k_w"):
        block.params[name] += 0.2 * torch.randn(block.params[name].shape, generator=g).cuda()
    x, dy = torch.randn(n, channels, generator=g).cuda(), torch.randn(n, channels, generator=g).cuda()
    y, kept = block.forward(grid, x, 7)
    grad, dx = block.backward(kept, dy)
    fvx.device_status()

    w = {name: p.double().cpu().requires_grad_() for name, p in block.params.items()}
    xd = x.double().cpu().requires_grad_()
    angle = _angles(block.rotary, grid.ijk())
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def turned(t, weight):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
        half = block.rotary.size // 2
        u, v = t[..., :half], t[..., half:2 * half]
        return torch.cat([u * cos - v * sin, v * cos + u * sin, t[..., 2 * half:]], -1)

    h = (xd - xd.mean(1, keepdim=True)) / (xd.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    qkv = ((h * w["norm_w"] + w["norm_b"]) @ w["qkv"]).view(n, 3 * heads, -1)
    q, k, v = turned(qkv[:, :heads], w["q_w"]), turned(qkv[:, heads:2 * heads], w["k_w"]), qkv[:, 2 * heads:]
    offsets, seen = [int(o) for o in grid.batch_offsets()], []
    for a, b in zip(offsets, offsets[1:]):
        s = torch.einsum("qhd,khd->hqk", q[a:b], k[a:b]) * q.shape[2] ** -0.5
        seen.append(torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v[a:b]))
    stays, scale = drawn(0, n * channels, 0.2, block.seed, 7)
    want_y = xd + (torch.cat(seen).reshape(n, -1) @ w["out"]) * torch.from_numpy(stays.reshape(n, channels) * scale)
    want = torch.autograd.grad(want_y, [xd] + list(w.values()), dy.double().cpu())
    pairs = [(y, want_y.detach(), "y"), (dx, want[0], "x")] + [(grad[m], t, m) for m, t in zip(w, want[1:])]
    for mine, value, name in pairs:
        assert (mine.double().cpu() - value).abs().max() <= 8e-4 * value.abs().max(), name


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_training_runs(dtype):
    from examples.voxel_attention import train

    losses = train(voxels=3000, channels=64, steps=3, dtype=getattr(torch, dtype))
    assert len(losses) == 3 and all(np.isfinite(losses))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_passes_repeat_bit_for_bit_and_captured(dtype):
    """No sum depends on the order in which blocks finish; a captured pass gives what the plain one does."""
    import sparse_convolution_gb300 as fvx
    from examples.voxel_attention import VoxelAttention

    dtype = getattr(torch, dtype)
    grid, g = _grid(4000, 2, 24, 5)
    block = VoxelAttention(64, 2, dtype)
    x = torch.randn(grid.n_active, 64, generator=g).cuda().to(dtype)
    dy = torch.randn(grid.n_active, 64, generator=g).cuda().to(dtype)
    grid.batch_offsets()  # read once, outside the capture

    def once():
        y, kept = block.forward(grid, x, 3)
        grad, dx = block.backward(kept, dy)
        return [y, dx, grad["q_w"], grad["k_w"], grad["norm_w"]]

    first = once()
    assert all(torch.equal(a, b) for a, b in zip(first, once()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once()
    x.add_(0.25)
    again = once()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, again))
    fvx.device_status()
