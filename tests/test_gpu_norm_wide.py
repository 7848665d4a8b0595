"""Layer norm and checkpoints of rows wider than 1024 channels, where a row
takes a block: widths, pitches and bases that allow accesses of two fp32 values
but not of four.  Definitions and tolerances are those of test_gpu_norm."""
import numpy as np
import pytest

from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu


def _fill_scratch(n):
    """A call that leaves values other than zero wherever the next one's
    partial sums may lie."""
    import sparse_convolution_gb300 as fvx

    x, w, _, dy = N._inputs(n, 65536, "f32", 3)
    _, mean, rstd = fvx.layer_norm(x, w)
    fvx.layer_norm_backward(dy, x, mean, rstd, w)


# (rows, channels, pitch padding, leading columns)
PAIRS = [(9, 1026, 0, 0), (7, 2046, 0, 0), (5, 3000, 2, 0), (6, 1028, 2, 0), (40, 2000, 4, 2), (2, 65534, 0, 0)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,c,pad,lead", PAIRS)
def test_checkpoint_bits_of_pairs(n, c, pad, lead, group):
    import torch

    import sparse_convolution_gb300 as fvx

    x, w, b, _ = N._inputs(n, c, "f32", n + c + group, pad, lead=lead)
    codes, steps = N._codes_ref(x.cpu().numpy(), group)
    held = N._held(codes, steps, group)
    for made in (lambda: fvx.Checkpoint8.pack(x, group=group), lambda: fvx.layer_norm(x, w, b, checkpoint_group=group)[3]):
        fill = [torch.full((n, c), 77, dtype=torch.int8, device="cuda") for _ in range(4)]
        del fill  # whatever is not written holds something else
        ck = made()
        assert np.array_equal(ck.codes.cpu().numpy(), codes)
        assert np.array_equal(ck.steps.cpu().numpy().view(np.uint32), steps.view(np.uint32))
        assert np.array_equal(ck.restore().cpu().numpy(), held)


@pytest.mark.parametrize("n,c,pad,lead", PAIRS)
def test_weight_gradients_of_pairs(n, c, pad, lead):
    """dweight and dbias of every channel, x from the tensor and from its codes."""
    import sparse_convolution_gb300 as fvx

    x, w, b, dy = N._inputs(n, c, "f32", n * 131 + c, pad, lead=lead)
    y, mean, rstd, ck = fvx.layer_norm(x, w, b, checkpoint_group=128)
    if c <= 16384:
        N._check_forward(y, mean, rstd, x, N._np(w), N._np(b), 1e-5, "f32")
    for source, xr in ((x, N._np(x)), (ck, N._np(ck.restore()))):
        _fill_scratch(n)
        dx, dw, db = fvx.layer_norm_backward(dy, source, mean, rstd, w)
        if c <= 16384:
            N._check_backward((dx, dw, db), dy, xr, mean, rstd, N._np(w), "f32")
        dyr, mr, rr = N._np(dy), N._np(mean)[:, None], N._np(rstd)[:, None]
        _, dwr, dbr = N._ref_backward(dyr, xr, mr, rr, N._np(w))
        xh, exh = np.abs((xr - mr) * rr), 4 * N.U * (np.abs(xr) + np.abs(mr)) * rr
        # fewer than 300 sums of at most n terms' parts, as in N._check_backward
        m, ay = n + 300, np.abs(dyr)
        N._close(N._np(dw), dwr, m * N.U * (ay * xh).sum(0) + (ay * exh).sum(0), "dweight")
        N._close(N._np(db), dbr, m * N.U * ay.sum(0), "dbias")
