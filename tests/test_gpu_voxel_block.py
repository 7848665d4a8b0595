"""The example that runs the operators together (examples/voxel_block.py): its
gradients against the formulas in 64 bits, and its losses."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _attend(q, k, v, qo, ko, mask):
    """Plain attention, differentiable; heads equal."""
    out = []
    for b in range(len(qo) - 1):
        qs, ks, vs = q[qo[b]:qo[b + 1]], k[ko[b]:ko[b + 1]], v[ko[b]:ko[b + 1]]
        if mask is not None:
            keep = mask[ko[b]:ko[b + 1]]
            ks, vs = ks[keep], vs[keep]
        if ks.shape[0] == 0:
            out.append(torch.zeros_like(qs))
            continue
        s = torch.einsum("qhd,khd->hqk", qs, ks) * q.shape[2] ** -0.5
        out.append(torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), vs))
    return torch.cat(out)


def test_gradients_match_the_formulas():
    """fp32 against autograd in 64 bits, with x's held values (8 bits) in place
    of x where the block reads them.

    Tolerance, of the largest value of each gradient: an fp32 sum of n terms
    wanders from the exact one by about sqrt(n) 2^-24 of its terms' root sum of
    squares; the longest sums here have 27 * 32 terms (conv) or 1500 (over the
    voxels), so about 40 * 6e-8 = 2.4e-6 per operator, and the chain has six of
    them.  Differences (softmax's and norm's gradients) lose up to a factor of
    about 30 where they nearly cancel: 6 * 30 * 2.4e-6 = 4e-4, taken as 5e-4."""
    import sparse_convolution_gb300 as fvx
    from examples.voxel_block import VoxelBlock

    g = torch.Generator().manual_seed(3)
    samples, channels, heads, lens = 3, 32, 2, (7, 0, 20)
    coords = torch.randint(0, 12, (1500, 3), dtype=torch.int32, generator=g).cuda()
    grid = fvx.Grid.build(coords, [0, 500, 900, 1500])
    kmap, kmap_t = fvx.KernelMap(grid, grid, 1), fvx.KernelMap(grid, grid, 1, transposed=True)
    so = [0, 7, 7, 27]
    mask = (torch.rand(27, generator=g) < 0.8).cuda()
    x = torch.randn(grid.n_active, channels, generator=g).cuda()
    block = VoxelBlock(channels, heads, sum(lens), samples, torch.float32, group=32)
    dreadout = torch.randn(samples, heads, channels // heads, generator=g).cuda()
    readout, kept = block.forward(grid, kmap, x, so, mask)
    grad, dx = block.backward(grid, kmap, kmap_t, so, mask, kept, dreadout)
    fvx.device_status()

    held = kept[4].restore().double().cpu()
    w = {n: p.double().cpu().requires_grad_() for n, p in block.params.items()}
    ii, oo, _ = (t.long().cpu() for t in kmap.pairs())
    po, vo = kmap.offsets, [int(v) for v in grid.batch_offsets()]
    mean, rstd = kept[2].double().cpu()[:, None], kept[3].double().cpu()[:, None]

    def passes(values, h_values):
        """The readouts; the conv's input is h_values where given."""
        h = (values - values.mean(1, keepdim=True)) / (values.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
        h = h * w["norm_w"] + w["norm_b"]
        if h_values is not None:
            h = h_values
        y = torch.zeros(len(h), channels, dtype=torch.float64)
        for s in range(27):
            a, b = int(po[s]), int(po[s + 1])
            y = y.index_add(0, oo[a:b], h[ii[a:b]] @ w["conv"][s])
        y = y.view(-1, heads, channels // heads)
        z = y + _attend(y, w["k"], w["v"], vo, so, mask.cpu())
        return h, _attend(w["query"], z, z, list(range(samples + 1)), vo, None)

    exact = x.double().cpu()
    h, want_readout = passes(exact, None)
    assert (readout.double().cpu() - want_readout).abs().max() <= 5e-4 * want_readout.abs().max()
    # the forward pass ran on x; its gradient up to the conv's input is that of the exact h
    h_leaf = h.detach().requires_grad_()
    _, r = passes(exact, h_leaf)
    names = ["k", "v", "query"]
    got = torch.autograd.grad(r, [h_leaf] + [w[n] for n in names], dreadout.double().cpu(), retain_graph=True)
    dh, want = got[0], dict(zip(names, got[1:]))
    # dy of the conv, then its weights' gradient from the held values
    h_held = (held - mean) * rstd * w["norm_w"].detach() + w["norm_b"].detach()
    y_leaf = torch.zeros(len(h), channels, dtype=torch.float64)
    for s in range(27):
        a, b = int(po[s]), int(po[s + 1])
        y_leaf = y_leaf.index_add(0, oo[a:b], h.detach()[ii[a:b]] @ w["conv"][s].detach())
    y_leaf.requires_grad_()
    y = y_leaf.view(-1, heads, channels // heads)
    z = y + _attend(y, w["k"].detach(), w["v"].detach(), vo, so, mask.cpu())
    r = _attend(w["query"].detach(), z, z, list(range(samples + 1)), vo, None)
    dy, = torch.autograd.grad(r, y_leaf, dreadout.double().cpu())
    want["conv"] = torch.stack([h_held[ii[int(po[s]):int(po[s + 1])]].T @ dy[oo[int(po[s]):int(po[s + 1])]]
                                for s in range(27)])
    # the norm's gradient at the held values, with the forward pass's statistics
    xh = (held - mean) * rstd
    gx = dh * w["norm_w"].detach()
    want["norm_w"], want["norm_b"] = (dh * xh).sum(0), dh.sum(0)
    want_dx = rstd * (gx - gx.mean(1, keepdim=True) - xh * (gx * xh).mean(1, keepdim=True))
    for name, value in list(want.items()) + [("x", want_dx)]:
        mine = (dx if name == "x" else grad[name]).double().cpu()
        assert (mine - value).abs().max() <= 5e-4 * value.abs().max(), name


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_training_lowers_the_loss(dtype):
    from examples.voxel_block import train

    losses = train(voxels=6000, channels=64, steps=4, dtype=getattr(torch, dtype))
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_passes_repeat_bit_for_bit(dtype):
    """No sum depends on the order in which blocks happen to finish, but those
    of the conv's weight gradient, which adds with atomics."""
    import sparse_convolution_gb300 as fvx
    from examples.voxel_block import VoxelBlock

    g = torch.Generator().manual_seed(5)
    dtype = getattr(torch, dtype)
    coords = torch.randint(0, 24, (9000, 3), dtype=torch.int32, generator=g).cuda()
    grid = fvx.Grid.build(coords, [0, 4000, 9000])
    kmap, kmap_t = fvx.KernelMap(grid, grid, 1), fvx.KernelMap(grid, grid, 1, transposed=True)
    so = [0, 200, 577]
    mask = (torch.rand(577, generator=g) < 0.9).cuda()
    x = torch.randn(grid.n_active, 64, generator=g).cuda().to(dtype)
    block = VoxelBlock(64, 4, 577, 2, dtype)
    dreadout = torch.randn(2, 4, 16, generator=g).cuda().to(dtype)

    def once():
        readout, kept = block.forward(grid, kmap, x, so, mask)
        grad, dx = block.backward(grid, kmap, kmap_t, so, mask, kept, dreadout)
        return [readout, dx] + [grad[n] for n in ("k", "v", "query", "norm_w", "norm_b")]

    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))
    fvx.device_status()
