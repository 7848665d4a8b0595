"""The C entry of the norm's backward pass with dx in dy's own memory: the
same bits as with a tensor of its own, for every kernel that serves a row."""
import ctypes

import pytest

from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,pad", [(700, 64, 0), (60, 1000, 0), (200_016, 64, 0), (200_016, 64, 8), (31, 179, 3),
                                     (9, 1026, 0), (11, 4096, 0), (5, 1101, 2)])
def test_dx_over_dy(n, c, pad, dtype, codes):
    import torch

    import sparse_convolution_gb300 as fvx

    x, w, b, dy = N._inputs(n, c, dtype, n + c, pad)
    wide = torch.zeros(n, c + pad, dtype=dy.dtype, device="cuda")
    wide[:, :c] = dy
    dy = wide[:, :c]
    _, mean, rstd, ck = fvx.layer_norm(x, w, b, checkpoint_group=64)
    at = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    source = (None, c, 64, at(ck.codes), at(ck.steps)) if codes else (at(x), c + pad, 0, None, None)

    def backward(dy, dx):
        dw, db = (torch.full((c,), float("nan"), device="cuda") for _ in range(2))
        assert fvx.load().fvx_layer_norm_backward(
            fvx.FVX_F32 if dtype == "f32" else fvx.FVX_BF16, at(dy), c + pad, *source, n, c, at(w), at(mean), at(rstd),
            at(dx), c + pad, at(dw), at(db), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        return dx, dw, db

    want = backward(dy, torch.zeros_like(wide)[:, :c])
    own = wide.clone()[:, :c]
    got = backward(own, own)
    for name, p, q in zip(("dx", "dweight", "dbias"), got, want):
        assert torch.equal(p, q), name
