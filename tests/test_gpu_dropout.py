"""Dropout against the generator's definition in numpy: what is kept bit for
bit, values in 64 bits.  A kept value x s is rounded once (the factor s once
more) and the sum with the residual once: 2 u |x s| + u |y|, u = 2^-24; bf16
results add half a step, 2^-8 of the value."""
import numpy as np
import pytest

from tests.gpu_common import BF16_OUT_REL
from tests.helpers_dropout import kept

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SEED, OFFSET = 0x123456789ABCDEF0, 0xFEDCBA9876543210


def _np(t):
    return t.detach().double().cpu().numpy()


def _rows(n, c, dtype, rng, pad=0, lead=0):
    base = torch.zeros(n, lead + c + pad, dtype=DT[dtype], device="cuda")
    x = base[:, lead:lead + c]
    x.copy_(torch.from_numpy(rng.normal(size=(n, c)) + 2.0))
    return x


def _check(y, x, residual, p, seed, offset, dtype):
    stays, scale = kept(0, x.numel(), p, seed, offset)
    xs = np.where(stays.reshape(x.shape), _np(x) * scale, 0.0)
    want = xs + (0 if residual is None else _np(residual))
    err = np.abs(_np(y) - want)
    bound = 2 * U * np.abs(xs) + (0 if residual is None else U * np.abs(want))
    if dtype == "bf16":
        bound = bound + BF16_OUT_REL * np.abs(want)
    assert np.all(err <= bound), float((err - bound).max())


# rows, values, padding, leading: one value; odd numbers; vectors of eight with and without gaps; bases and pitches that
# no vector reads; pitches around the limits of the division
SHAPES = [(1, 1, 0, 0), (1, 7, 0, 0), (1, 8, 0, 0), (1, 9, 0, 0), (1, 256, 0, 0), (300, 1, 0, 0), (300, 1, 1, 0), (257, 2, 3, 1),
          (513, 7, 0, 0), (513, 7, 1, 0), (100, 8, 8, 0), (100, 8, 0, 0), (99, 24, 8, 8), (99, 24, 1, 0), (77, 101, 0, 0),
          (77, 101, 33, 0), (50, 128, 8, 0), (50, 128, 0, 0), (31, 255, 1, 1), (31, 256, 4, 0), (13, 511, 2, 0), (13, 512, 2, 0),
          (13, 513, 2, 1), (3, 70001, 3, 0), (2, 70008, 8, 8), (20011, 32, 0, 0), (5000, 36, 0, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,pad,lead", SHAPES)
def test_forward_and_backward(n, c, pad, lead, dtype):
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(n * 31 + c)
    x, r, dy = _rows(n, c, dtype, rng, pad, lead), _rows(n, c, dtype, rng), _rows(n, c, dtype, rng, pad)
    for p in (0.1, 0.5):
        _check(fvx.dropout(x, p, SEED, OFFSET), x, None, p, SEED, OFFSET, dtype)
        _check(fvx.dropout(x, p, SEED, OFFSET, residual=r), x, r, p, SEED, OFFSET, dtype)
        _check(fvx.dropout_backward(dy, p, SEED, OFFSET), dy, None, p, SEED, OFFSET, dtype)
    fvx.device_status()


@pytest.mark.parametrize("seed,offset", [(0, 0), (1, 0), (0, 1), (2 ** 64 - 1, 2 ** 64 - 1), (2 ** 63, 2 ** 32)])
def test_seeds_and_offsets(seed, offset):
    import sparse_convolution_gb300 as fvx

    x = _rows(64, 40, "f32", np.random.default_rng(1))
    _check(fvx.dropout(x, 0.3, seed, offset), x, None, 0.3, seed, offset, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_and_everything_dropped(dtype):
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(2)
    for shape in ((65, 40), (65, 41)):
        x, r = _rows(*shape, dtype, rng), _rows(*shape, dtype, rng)
        x[3, 5], x[4, 6] = float("nan"), float("inf")
        assert torch.equal(fvx.dropout(x, 0.0, 1).nan_to_num(7.0), x.nan_to_num(7.0))
        assert torch.equal(fvx.dropout(x, 1.0, 1, residual=r), r)  # dropped, whatever they were
        assert not fvx.dropout(x, 1.0, 1).any()
        assert torch.equal(fvx.dropout(x, 2.0 ** -18, 1).nan_to_num(7.0), x.nan_to_num(7.0))  # below half of 2^-16


def test_any_shape_and_memory():
    """The same bits whatever the strides: three dimensions, one value, none, a transposed tensor."""
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(size=(17, 6, 40))).float().cuda()
    y = fvx.dropout(x, 0.4, 5, 6)
    _check(y, x, None, 0.4, 5, 6, "f32")
    assert torch.equal(fvx.dropout(x.view(-1), 0.4, 5, 6), y.view(-1))
    assert torch.equal(fvx.dropout(x.transpose(0, 2).contiguous().transpose(0, 2), 0.4, 5, 6), y)
    assert torch.equal(fvx.dropout(x[0].t(), 0.4, 5, 6), fvx.dropout(x[0].t().contiguous(), 0.4, 5, 6))
    assert torch.equal(fvx.dropout(x[:, 0], 0.4, 5, 6), fvx.dropout(x[:, 0].contiguous(), 0.4, 5, 6))
    assert torch.equal(fvx.dropout(x[:1, :1, :1].expand(4, 5, 6), 0.4, 5, 6),
                       fvx.dropout(x[:1, :1, :1].expand(4, 5, 6).contiguous(), 0.4, 5, 6))
    one = torch.tensor(3.0, device="cuda")
    _check(fvx.dropout(one, 0.4, 5, 6).view(1), one.view(1), None, 0.4, 5, 6, "f32")
    for shape in ((0,), (0, 8), (8, 0), (3, 0, 2)):
        assert fvx.dropout(torch.empty(shape, device="cuda"), 0.4, 5).shape == shape


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("c,pad", [(64, 0), (64, 8), (37, 0), (37, 2)])
def test_in_place(c, pad, dtype):
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(4)
    x, r = _rows(200, c, dtype, rng, pad), _rows(200, c, dtype, rng, pad)
    want = fvx.dropout(x, 0.2, 9, 1, residual=r)
    x2, r2 = _rows(200, c, dtype, np.random.default_rng(0), pad), _rows(200, c, dtype, np.random.default_rng(0), pad)
    x2.copy_(x)
    r2.copy_(r)
    assert torch.equal(fvx.dropout(x2, 0.2, 9, 1, residual=r, out=x2), want) and torch.equal(x2, want)
    assert torch.equal(fvx.dropout(x, 0.2, 9, 1, residual=r2, out=r2), want) and torch.equal(r2, want)
    if pad:  # what lies between the rows stays
        assert not r2.as_strided((200, pad), (c + pad, 1), r2.storage_offset() + c)[:-1].any()


def test_state_on_the_device_and_captured():
    """A captured call draws anew when the state's values change between replays."""
    import sparse_convolution_gb300 as fvx

    x = _rows(300, 40, "bf16", np.random.default_rng(5))
    as_int64 = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    state = torch.tensor([as_int64(2 ** 63 + 11), 7], device="cuda")
    assert torch.equal(fvx.dropout(x, 0.3, state, 5), fvx.dropout(x, 0.3, 2 ** 63 + 11, 12))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fvx.dropout(x, 0.3, state)
        dx = fvx.dropout_backward(x, 0.3, state)
        state[1] += 1
    for offset in (7, 8, 9):
        graph.replay()
        torch.cuda.synchronize()
        want = fvx.dropout(x, 0.3, 2 ** 63 + 11, offset)
        assert torch.equal(y, want) and torch.equal(dx, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fvx.dropout(x, 0.3, 4, stream=side)
    side.synchronize()
    assert torch.equal(got, fvx.dropout(x, 0.3, 4))


def test_places_past_32_bits():
    """The last values of a tensor of 2^32 + 1000: their counters, addresses and rows."""
    import sparse_convolution_gb300 as fvx

    n = (1 << 32) + 1000
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = fvx.dropout(x, 0.5, 3, 4)
    first = n - 2000
    first -= first % 8
    stays, scale = kept(first, n - first, 0.5, 3, 4)
    assert np.array_equal(_np(y[first:]), np.where(stays, scale, 0.0))
    # rows with a gap: the same values by another kernel
    z = x[:(1 << 32)].view(-1, 1 << 20)[:, :(1 << 20) - 24]
    w = fvx.dropout(z, 0.5, 3, 4, out=y[:(1 << 32)].view(-1, 1 << 20)[:, :(1 << 20) - 24])
    count = (1 << 20) - 24
    stays, scale = kept(4095 * count, count, 0.5, 3, 4)
    assert np.array_equal(_np(w[-1]), np.where(stays, scale, 0.0))
    # a base that no vector reads: the kernel of any alignment
    y = fvx.dropout(x[1:], 0.5, 3, 4)
    stays, scale = kept(first, n - 1 - first, 0.5, 3, 4)
    assert np.array_equal(_np(y[first:]), np.where(stays, scale, 0.0))


def test_refusals():
    import sparse_convolution_gb300 as fvx

    x = torch.zeros(6, 16, device="cuda")
    state = torch.zeros(2, dtype=torch.int64, device="cuda")
    for call in (lambda: fvx.dropout(x.half(), 0.1, 1), lambda: fvx.dropout(x.cpu(), 0.1, 1), lambda: fvx.dropout(x, -0.1, 1),
                 lambda: fvx.dropout(x, 1.1, 1), lambda: fvx.dropout(x, float("nan"), 1), lambda: fvx.dropout(x, 0.1, -1),
                 lambda: fvx.dropout(x, 0.1, 1 << 64), lambda: fvx.dropout(x, 0.1, 1, -1),
                 lambda: fvx.dropout(x, 0.1, 1, residual=x[:5]), lambda: fvx.dropout(x, 0.1, 1, residual=x.bfloat16()),
                 lambda: fvx.dropout(x, 0.1, 1, residual=x.cpu()), lambda: fvx.dropout(x, 0.1, state.int()),
                 lambda: fvx.dropout(x, 0.1, state[:1]), lambda: fvx.dropout(x, 0.1, state.cpu()),
                 lambda: fvx.dropout(x, 0.1, 1, out=x[:5]), lambda: fvx.dropout(x, 0.1, 1, out=x.bfloat16()),
                 lambda: fvx.dropout(x[:, :8], 0.1, 1, out=x[:, ::2]), lambda: fvx.dropout_backward(x, 2.0, 1)):
        with pytest.raises(fvx.FvxError) as e:
            call()
        assert e.value.status == "FVX_ERR_INVALID_ARG"
