"""A Checkpoint8 whose parts do not belong together is refused by every call
that reads it, before any CUDA work (no GPU needed): the kernels would read
past the steps' end."""
import pytest
import torch

import sparse_convolution_gb300 as fvx


def _parts(codes=(6, 100), steps=(6, 4), group=32, code_type=torch.int8, step_type=torch.float32):
    return fvx.Checkpoint8(torch.zeros(codes, dtype=code_type), torch.ones(steps, dtype=step_type), group, torch.float32)


def _strided(name):
    ck = _parts()
    setattr(ck, name, getattr(ck, name).t().contiguous().t())
    return ck


@pytest.mark.parametrize("ck,named", [
    (_parts(steps=(6, 1)), "steps"), (_parts(steps=(5, 4)), "steps"), (_parts(steps=(24,)), "steps"),
    (_parts(group=64), "steps"), (_parts(step_type=torch.float64), "steps"), (_parts(group=16), "group"),
    (_parts(group=0), "group"), (_parts(code_type=torch.uint8), "codes"), (_parts(codes=(600,), steps=(600, 1)), "codes"),
    (_strided("codes"), "codes"), (_strided("steps"), "steps")])
def test_parts_that_do_not_belong_together(ck, named):
    dy, row, out = torch.zeros(6, 100), torch.ones(6), torch.zeros(6, 100)
    calls = [lambda: ck.restore(), lambda: ck.restore(out=out), lambda: ck.layer_norm(row, row)]
    if tuple(ck.shape) == (6, 100):  # another shape than dy's is refused for that
        calls.append(lambda: fvx.layer_norm_backward(dy, ck, row, row))
    for call in calls:
        with pytest.raises(fvx.FvxError, match=named) as e:
            call()
        assert e.value.status == "FVX_ERR_INVALID_ARG"
