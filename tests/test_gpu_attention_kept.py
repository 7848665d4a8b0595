"""What the forward pass returned, kept by the caller in memory of its own:
the backward pass takes it wherever its elements lie."""
import pytest

from tests import test_gpu_attention as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,d", [(1, 3), (3, 20), (2, 64)])
def test_out_at_any_element(heads, d, dtype):
    import torch

    import sparse_convolution_gb300 as fvx

    t, qo, ko, mask = A._case([40, 9], [33, 60], heads, 1, d, dtype, d, 0.2)
    want = A._run(t, qo, ko, mask)
    room = torch.empty(want["out"].numel() + 1, dtype=want["out"].dtype, device="cuda")
    kept = room[1:].view_as(want["out"])
    kept.copy_(want["out"])
    assert kept.data_ptr() % 16
    lse = torch.empty(want["lse"].numel() + 1, device="cuda")[1:].view_as(want["lse"])
    lse.copy_(want["lse"])
    got = fvx.cross_attention_backward(t["dout"], t["q"], t["k"], t["v"], kept, lse, qo, ko, key_mask=mask)
    for n, g in zip(("dq", "dk", "dv"), got):
        assert torch.equal(g, want[n]), n
