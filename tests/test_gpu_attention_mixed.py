"""The backward pass of batches whose samples are cut in different ways: many
rows on few keys beside few rows on many keys, samples of neither.  Definitions
and tolerances are those of test_gpu_attention."""
import pytest

from tests import test_gpu_attention as A
from tests.test_gpu_failures import CountingAllocator

pytestmark = pytest.mark.gpu


class PeakAllocator(CountingAllocator):
    peak = 0

    def _alloc(self, nbytes, stream, ctx):
        p = super()._alloc(nbytes, stream, ctx)
        self.peak = max(self.peak, sum(self.live.values()))
        return p


@pytest.mark.parametrize("d,heads,kv_heads", [(128, 1, 1), (64, 1, 1), (64, 6, 2), (96, 2, 2)])
@pytest.mark.parametrize("qlens,klens", [([20000, 100], [100, 20000]), ([0, 90, 6000, 7, 1], [50, 9000, 128, 0, 400]),
                                         ([129, 10000, 300], [8000, 130, 300])])
def test_samples_cut_in_different_ways(qlens, klens, d, heads, kv_heads):
    t, qo, ko, mask = A._case(qlens, klens, heads, kv_heads, d, "bf16", sum(qlens) + d, 0.1)
    got = A._check(t, qo, ko, mask)
    again = A._run(t, qo, ko, mask)
    assert all((got[n] == again[n]).all() for n in got)


def test_a_sample_pays_for_its_own_cut():
    """Partial sums are kept for the samples that need them.  20,000 rows on 100
    keys need at most one slab of dK and of dV per multiprocessor (157 row
    tiles, one key tile), 100 rows on 20,000 keys one of dQ; a slab is 128 x 128
    fp32 values, 64 KiB, and memory is taken 32 MiB at least at a time: dQ's 9.5
    MiB with dK's and the statistics in one piece, dV's in another."""
    t, qo, ko, _ = A._case([20000, 100], [100, 20000], 1, 1, 128, "bf16", 5)
    with PeakAllocator() as memory:
        A._run(t, qo, ko, None)
    assert memory.calls > 0 and not memory.live
    assert memory.peak <= 3 * (32 << 20), memory.peak
