"""Norm calls from several host threads, each on its own stream, whose rows
take the same kernel with different amounts of shared memory."""
import ctypes
import threading

import pytest

from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu


def test_threads_with_stages_of_different_sizes():
    import torch

    import sparse_convolution_gb300 as fvx

    f, at = fvx.load().fvx_layer_norm, lambda t: ctypes.c_void_p(t.data_ptr())
    calls, want = [], []
    # 8 lanes of 16 bytes each, streamed in stages of 10, 8 and 9 KB
    for c in (40, 64, 48):
        x, w, b, _ = N._inputs(330_000, c, "bf16", c)
        want.append(fvx.layer_norm(x, w, b))
        for _ in range(2):
            side, out = torch.cuda.Stream(), [torch.empty_like(t) for t in want[-1]]
            n = x.shape[0]
            calls.append((side, (x, w, b), out, len(want) - 1,
                          (fvx.FVX_BF16, at(x), c, n, c, at(w), at(b), 1e-5, at(out[0]), c, at(out[1]), at(out[2]), 0,
                           None, None, ctypes.c_void_p(side.cuda_stream))))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(calls))

    def work(args):
        start.wait()
        for _ in range(4000):
            if f(*args):
                failed.append(fvx.load().fvx_last_error())
                return

    threads = [threading.Thread(target=work, args=(call[-1],)) for call in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for _, _, out, i, _ in calls:
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))
