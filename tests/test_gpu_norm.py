"""Layer norm (forward, backward) and 8-bit activation checkpoints against
plain implementations in 64 bits (the checkpoint's codes against the same fp32
operations in numpy, bit for bit).

Tolerances.  u = 2^-24 is half an ulp of fp32 relative to 1.  A sum of m terms
in any order is within (m - 1) u sum|terms|; the kernels add at most 37 values
in a row of up to 1024 (32 in a lane, 5 steps across lanes) and 64 + 8 + 8 of a
wider one up to 16384, so K = 64 / 128 covers the mean, the deviation and the
final operations.  bf16 results add their rounding (BF16_OUT_REL of the value).
"""
import numpy as np
import pytest

from tests.gpu_common import BF16_OUT_REL

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": "float32", "bf16": "bfloat16"}


def _t(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(getattr(torch, DT[dtype]))


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(n, c, dtype, seed, pad=0, offset=0.5, lead=0):
    import torch

    rng = np.random.default_rng(seed)
    base = torch.zeros(n, lead + c + pad, dtype=getattr(torch, DT[dtype]), device="cuda")
    base[:, lead:lead + c] = _t(rng.normal(size=(n, c)) * np.exp(rng.normal(size=c)) + offset, dtype)
    w, b = _t(1 + 0.2 * rng.normal(size=c), "f32"), _t(rng.normal(size=c), "f32")
    return base[:, lead:lead + c], w, b, _t(rng.normal(size=(n, c)), dtype)


def _ref_forward(x, w, b, eps):
    mean = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    return (x - mean) * rstd * w + b, mean, rstd


def _ref_backward(dy, x, mean, rstd, w):
    xh = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def _close(got, want, bound, what):
    err = np.abs(got - want)
    assert np.all(err <= bound), (what, float((err - bound).max()), float(err.max()))


def _k(c):
    return 64 if c <= 1024 else 128


def _check_forward(y, mean, rstd, x, w, b, eps, dtype):
    xr = _np(x)
    c = xr.shape[1]
    yr, mr, rr = _ref_forward(xr, w, b, eps)
    size = np.abs(xr).max(1, keepdims=True) + np.abs(mr)
    _close(_np(mean)[:, None], mr, _k(c) * U * size, "mean")
    # d rstd / rstd = -dvar / (2 (var + eps)); dvar <= K u (var + 2 |d mean| size)
    _close(_np(rstd)[:, None], rr, rr * _k(c) * U * (1 + size ** 2 * rr ** 2), "rstd")
    bound = _k(c) * U * (size * rr * np.abs(w) * (1 + size * rr) + np.abs(b) + np.abs(yr))
    _close(_np(y), yr, bound + (BF16_OUT_REL * np.abs(yr) if dtype == "bf16" else 0), "y")


def _check_backward(got, dy, x, mean, rstd, w, dtype):
    dyr, xr, mr, rr = _np(dy), x, _np(mean)[:, None], _np(rstd)[:, None]
    n, c = dyr.shape
    dxr, dwr, dbr = _ref_backward(dyr, xr, mr, rr, w)
    g, xh = np.abs(dyr * w), np.abs((xr - mr) * rr)
    exh = 4 * U * (np.abs(xr) + np.abs(mr)) * rr  # of xh itself
    scale = rr * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
    more = rr * (exh * (g * xh).mean(1, keepdims=True) + xh * (g * exh).mean(1, keepdims=True))
    _close(_np(got[0]), dxr, _k(c) * U * scale + more + (BF16_OUT_REL * np.abs(dxr) if dtype == "bf16" else 0), "dx")
    # a lane adds its rows one after the other, then blocks and parts: fewer than n + 300 in all, and 512 here
    m = min(n, 512) + 300
    ay = np.abs(dyr)
    _close(_np(got[1]), dwr, m * U * (ay * xh).sum(0) + (ay * exh).sum(0), "dweight")
    _close(_np(got[2]), dbr, m * U * ay.sum(0), "dbias")


# (rows, channels, pitch padding, leading columns): one row, odd channel
# counts, pitches and bases that allow 16-, 4- and 2-byte accesses, widths at
# the edges of each kernel (a lane's vector, a warp's 32 vectors, 1024 values)
SHAPES = [(1, 256, 0, 0), (1, 1, 0, 0), (3, 2, 0, 0), (257, 7, 0, 0), (1000, 8, 0, 0), (513, 16, 0, 0), (400, 31, 2, 1),
          (700, 64, 0, 0), (700, 64, 8, 8), (700, 64, 3, 1), (300, 100, 33, 0), (65, 127, 0, 0), (50, 128, 4, 2),
          (129, 256, 0, 0), (90, 264, 0, 0), (33, 511, 0, 0), (64, 512, 0, 0), (40, 1000, 0, 0), (17, 1022, 2, 0),
          (21, 1023, 0, 0), (20, 1024, 0, 0), (9, 1025, 0, 0), (7, 1032, 8, 0), (5, 4100, 0, 0), (2, 16384, 0, 0),
          (5000, 24, 0, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,pad,lead", SHAPES)
def test_forward_and_backward(n, c, pad, lead, dtype):
    import sparse_convolution_gb300 as fvx

    x, w, b, dy = _inputs(n, c, dtype, n * 131 + c, pad, lead=lead)
    y, mean, rstd = fvx.layer_norm(x, w, b, eps=1e-5)
    _check_forward(y, mean, rstd, x, _np(w), _np(b), 1e-5, dtype)
    got = fvx.layer_norm_backward(dy, x, mean, rstd, w)
    _check_backward(got, dy, _np(x), mean, rstd, _np(w), dtype)
    again = fvx.layer_norm_backward(dy, x, mean, rstd, w)
    assert all((p == q).all() for p, q in zip(got, again))  # the sums' order is fixed


@pytest.mark.parametrize("c", [48, 2000])
def test_without_weight_and_bias(c):
    import sparse_convolution_gb300 as fvx

    x, _, _, dy = _inputs(70, c, "f32", 5)
    y, mean, rstd = fvx.layer_norm(x)
    _check_forward(y, mean, rstd, x, np.ones(c), np.zeros(c), 1e-5, "f32")
    _check_backward(fvx.layer_norm_backward(dy, x, mean, rstd), dy, _np(x), mean, rstd, np.ones(c), "f32")


def test_no_rows():
    import torch

    import sparse_convolution_gb300 as fvx

    x = torch.empty(0, 40, device="cuda")
    y, mean, rstd, ck = fvx.layer_norm(x, checkpoint_group=32)
    assert y.shape == (0, 40) and mean.shape == (0,) and ck.restore().shape == (0, 40)
    dx, dw, db = fvx.layer_norm_backward(x, ck, mean, rstd)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


def test_gradients_against_differences():
    """Central differences of the definition in 64 bits along random
    directions: h = 1e-4 leaves a truncation of about h^2 and a rounding of
    about 1e-16 / h, both far below the fp32 gradient's own error."""
    import sparse_convolution_gb300 as fvx

    n, c = 37, 50
    x, w, b, dy = _inputs(n, c, "f32", 11)
    _, mean, rstd = fvx.layer_norm(x, w, b)
    dx, dw, db = (_np(t) for t in fvx.layer_norm_backward(dy, x, mean, rstd, w))
    X, Wt, Bt, D = _np(x), _np(w), _np(b), _np(dy)
    f = lambda x_, w_, b_: float((_ref_forward(x_, w_, b_, 1e-5)[0] * D).sum())  # noqa: E731
    rng = np.random.default_rng(3)
    h = 1e-4
    for _ in range(4):
        ux, uw, ub = rng.normal(size=X.shape), rng.normal(size=c), rng.normal(size=c)
        num = (f(X + h * ux, Wt + h * uw, Bt + h * ub) - f(X - h * ux, Wt - h * uw, Bt - h * ub)) / (2 * h)
        ana = (dx * ux).sum() + (dw * uw).sum() + (db * ub).sum()
        size = np.abs(dx * ux).sum() + np.abs(dw * uw).sum() + np.abs(db * ub).sum()
        assert abs(num - ana) <= 1e-5 * size


def test_a_row_that_is_not_finite_stays_alone():
    import torch

    import sparse_convolution_gb300 as fvx

    x, w, b, _ = _inputs(40, 64, "bf16", 4)
    x[7, 3], x[9, 5] = float("nan"), float("inf")
    y, mean, rstd = fvx.layer_norm(x, w, b)
    bad = ~torch.isfinite(y.float()).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 9]


def test_constant_rows():
    """No spread: y is the bias, rstd 1 / sqrt(eps)."""
    import torch

    import sparse_convolution_gb300 as fvx

    x = torch.full((5, 96), 3.0, device="cuda")
    b = torch.arange(96.0, device="cuda")
    y, mean, rstd = fvx.layer_norm(x, None, b, eps=1e-3)
    assert (y == b).all() and (mean == 3).all()
    assert np.allclose(_np(rstd), 1e-3 ** -0.5, rtol=1e-6)


# ---------------------------------------------------------------- checkpoints
def _codes_ref(x, group):
    """The definition in numpy's fp32 (each operation rounded once)."""
    x = np.asarray(x, np.float32)
    n, c = x.shape
    g = -(-c // group)
    codes, steps = np.zeros((n, c), np.int8), np.zeros((n, g), np.float32)
    for j in range(g):
        part = x[:, j * group:(j + 1) * group]
        top = np.abs(part).max(1) if part.size else np.zeros(n, np.float32)
        fine = np.isfinite(top)
        held = fine & (top >= np.float32(2.0 ** -100))
        safe = np.where(held, top, np.float32(1)).astype(np.float32)
        inv = np.where(held, np.float32(127) / safe, np.float32(0)).astype(np.float32)
        with np.errstate(invalid="ignore"):
            q = np.rint((part * inv[:, None]).astype(np.float32))
        codes[:, j * group:(j + 1) * group] = np.where(held[:, None], q, 0).astype(np.int8)
        steps[:, j] = np.where(held, (top / np.float32(127)).astype(np.float32),
                               np.where(fine, np.float32(0), np.float32(np.nan)))
    return codes, steps


def _held(codes, steps, group):
    return (codes.astype(np.float32) * np.repeat(steps, group, 1)[:, :codes.shape[1]]).astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,c,pad,lead", [(1, 1, 0, 0), (5, 33, 0, 0), (300, 48, 0, 0), (200, 32, 8, 0), (77, 128, 0, 0),
                                          (50, 250, 6, 0), (64, 256, 3, 1), (31, 1000, 0, 0), (9, 1500, 0, 0),
                                          (7, 1101, 0, 0)])
def test_checkpoint_bits(n, c, pad, lead, group, dtype):
    """pack, the norm's own checkpoint and restore, bit for bit."""
    import torch

    import sparse_convolution_gb300 as fvx

    x, w, b, _ = _inputs(n, c, dtype, 7 * n + c + group, pad, lead=lead)
    xr = x.float().cpu().numpy()
    codes, steps = _codes_ref(xr, group)
    for ck in (fvx.Checkpoint8.pack(x, group=group), fvx.layer_norm(x, w, b, checkpoint_group=group)[3]):
        assert np.array_equal(ck.codes.cpu().numpy(), codes)
        assert np.array_equal(ck.steps.cpu().numpy().view(np.uint32), steps.view(np.uint32))
        held = _held(codes, steps, group)
        assert np.array_equal(ck.restore(torch.float32).cpu().numpy(), held)
        assert torch.equal(ck.restore().cpu(), torch.from_numpy(held).to(x.dtype))
    # within half a step of the activation: the product's rounding moves a code by at most 127 * 2^-23
    assert np.all(np.abs(held - xr) <= np.repeat(steps, group, 1)[:, :c] * (0.5 + 127 * 2.0 ** -22))


def test_checkpoint_quotients():
    """step = top / 127 and x (127 / top) as the fp32 division rounds them, for
    two million maxima over the whole range of magnitudes, both ends included."""
    import torch

    import sparse_convolution_gb300 as fvx

    g = torch.Generator(device="cuda").manual_seed(5)
    bits = torch.randint(0x0D800000, 0x7F800000, (1 << 21,), generator=g, device="cuda", dtype=torch.int32)
    bits[:4] = torch.tensor([0x0D800000, 0x0D800001, 0x7F7FFFFF, 0x7E800000], dtype=torch.int32)
    top = bits.view(torch.float32)
    x = top[:, None] * torch.rand(1 << 21, 32, generator=g, device="cuda")
    x[:, 7] = -top
    ck = fvx.Checkpoint8.pack(x, group=32)
    most = torch.full_like(top, 127.0)
    assert torch.equal(ck.steps[:, 0], top / most)
    assert torch.equal(ck.codes, torch.round(x * (most / top)[:, None]).to(torch.int8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_checkpoint_special_values(dtype):
    import torch

    import sparse_convolution_gb300 as fvx

    x = torch.zeros(6, 64, device="cuda", dtype=getattr(torch, DT[dtype]))
    x[1, 3], x[2, 40] = float("inf"), float("nan")
    x[3, :32], x[3, 32:] = 2.0 ** -101, 2.0 ** -99
    x[4, 0], x[5, 1] = -127.0, 2.0 ** 127
    held = fvx.Checkpoint8.pack(x, group=32).restore().float().cpu().numpy()
    assert not held[0].any()
    assert np.isnan(held[1, :32]).all() and not held[1, 32:].any()
    assert not held[2, :32].any() and np.isnan(held[2, 32:]).all()
    assert not held[3, :32].any() and np.allclose(held[3, 32:], 2.0 ** -99, rtol=2.0 ** -8)
    assert held[4, 0] == -127 and held[4, 1:].any() == False  # noqa: E712
    assert np.isclose(held[5, 1], 2.0 ** 127, rtol=2.0 ** -8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,group", [(1, 64, 64), (333, 100, 32), (200, 256, 64), (75, 33, 128), (40, 1024, 128),
                                       (11, 1500, 64)])
def test_backward_from_checkpoint(n, c, group, dtype):
    """The norm's backward pass and the recomputed output, x read from its codes."""
    import sparse_convolution_gb300 as fvx

    x, w, b, dy = _inputs(n, c, dtype, 17 * n + c)
    y, mean, rstd, ck = fvx.layer_norm(x, w, b, checkpoint_group=group)
    plain = fvx.layer_norm(x, w, b)
    assert all((p == q).all() for p, q in zip((y, mean, rstd), plain))
    held = _held(ck.codes.cpu().numpy(), ck.steps.cpu().numpy(), group).astype(np.float64)
    _check_backward(fvx.layer_norm_backward(dy, ck, mean, rstd, w), dy, held, mean, rstd, _np(w), dtype)
    m, r, wr, br = _np(mean)[:, None], _np(rstd)[:, None], _np(w), _np(b)
    want = (held - m) * r * wr + br
    bound = 8 * U * ((np.abs(held) + np.abs(m)) * r * np.abs(wr) + np.abs(br) + np.abs(want))
    _close(_np(ck.layer_norm(mean, rstd, w, b)), want, bound + (BF16_OUT_REL * np.abs(want) if dtype == "bf16" else 0),
           "again")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,group", [(300_003, 8, 32), (200_011, 64, 32), (150_001, 256, 64), (300_017, 48, 128),
                                       (60_007, 504, 64), (50_021, 1024, 128)])
def test_long_tensors(n, c, group, dtype):
    """Lengths that take the streaming kernels, with a last stage that is not
    full: rows from every part against the definitions, dweight and dbias
    against sums in 64 bits."""
    import torch

    import sparse_convolution_gb300 as fvx

    x, w, b, dy = _inputs(n, c, dtype, c)
    y, mean, rstd, ck = fvx.layer_norm(x, w, b, checkpoint_group=group)
    plain = fvx.layer_norm(x, w, b)
    assert all(torch.equal(p, q) for p, q in zip(plain, (y, mean, rstd)))
    packed = fvx.Checkpoint8.pack(x, group=group)
    assert torch.equal(packed.codes, ck.codes) and torch.equal(packed.steps, ck.steps)
    restored, again = ck.restore(torch.float32), ck.layer_norm(mean, rstd, w, b)
    at = torch.cat([torch.arange(0, 70), torch.arange(n // 2, n // 2 + 70), torch.arange(n - 600, n)]).cuda()
    xs = x[at]
    _check_forward(y[at], mean[at], rstd[at], xs, _np(w), _np(b), 1e-5, dtype)
    codes, steps = _codes_ref(xs.float().cpu().numpy(), group)
    held = _held(codes, steps, group)
    assert np.array_equal(ck.codes[at].cpu().numpy(), codes) and np.array_equal(ck.steps[at].cpu().numpy(), steps)
    assert np.array_equal(restored[at].cpu().numpy(), held)
    m, r, wr, br = _np(mean[at])[:, None], _np(rstd[at])[:, None], _np(w), _np(b)
    want = (held - m) * r * wr + br
    bound = 8 * U * ((np.abs(held) + np.abs(m)) * r * np.abs(wr) + np.abs(br) + np.abs(want))
    _close(_np(again[at]), want, bound + (BF16_OUT_REL * np.abs(want) if dtype == "bf16" else 0), "again")
    for source, xr in ((x, _np(xs)), (ck, held.astype(np.float64))):
        got = fvx.layer_norm_backward(dy, source, mean, rstd, w)
        fvx.device_status()
        repeat = fvx.layer_norm_backward(dy, source, mean, rstd, w)
        assert all(torch.equal(p, q) for p, q in zip(got, repeat))
        dyr = _np(dy[at])
        dxr = _ref_backward(dyr, xr, m, r, wr)[0]
        g, xh = np.abs(dyr * wr), np.abs((xr - m) * r)
        exh = 4 * U * (np.abs(xr) + np.abs(m)) * r
        scale = r * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
        more = r * (exh * (g * xh).mean(1, keepdims=True) + xh * (g * exh).mean(1, keepdims=True))
        _close(_np(got[0][at]), dxr, _k(c) * U * scale + more + (BF16_OUT_REL * np.abs(dxr) if dtype == "bf16" else 0), "dx")
        full = (source.float() if source is x else restored).double()
        xh = (full - mean.double()[:, None]) * rstd.double()[:, None]
        ex = 4 * U * (full.abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]
        d = dy.double()
        # rows of a lane one after the other, then groups, blocks and parts: at most n / 128 + 800 here
        bound = (n / 128 + 800) * U
        _close(_np(got[1]), _np((d * xh).sum(0)), bound * _np((d * xh).abs().sum(0)) + _np((d.abs() * ex).sum(0)), "dweight")
        _close(_np(got[2]), _np(d.sum(0)), bound * _np(d.abs().sum(0)), "dbias")


def test_another_stream():
    """Inputs made on one stream, the calls on another that waits for it."""
    import torch

    import sparse_convolution_gb300 as fvx

    x, w, b, dy = _inputs(20000, 64, "bf16", 8)
    want = fvx.layer_norm(x, w, b, checkpoint_group=64)
    wb = fvx.layer_norm_backward(dy, want[3], want[1], want[2], w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fvx.layer_norm(x, w, b, checkpoint_group=64, stream=side)
    gb = fvx.layer_norm_backward(dy, got[3], got[1], got[2], w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[3].codes, want[3].codes)
    assert all(torch.equal(p, q) for p, q in zip(gb, wb))


def test_large_offsets():
    """More than 2^31 values: the last rows are right."""
    import torch

    import sparse_convolution_gb300 as fvx

    n, c = (1 << 31) // 256 + 3, 256
    x = torch.zeros(n, c, device="cuda", dtype=torch.bfloat16)
    tail, w, b, _ = _inputs(3, c, "bf16", 21)
    x[-3:] = tail
    y, mean, rstd, ck = fvx.layer_norm(x, w, b, checkpoint_group=64)
    _check_forward(y[-3:], mean[-3:], rstd[-3:], tail, _np(w), _np(b), 1e-5, "bf16")
    codes, steps = _codes_ref(tail.float().cpu().numpy(), 64)
    assert np.array_equal(ck.codes[-3:].cpu().numpy(), codes)
    dx, _, _ = fvx.layer_norm_backward(y, ck, mean, rstd, w)
    held = _held(codes, steps, 64).astype(np.float64)
    want = _ref_backward(_np(y[-3:]), held, _np(mean[-3:])[:, None], _np(rstd[-3:])[:, None], _np(w))[0]
    assert np.allclose(_np(dx[-3:]), want, rtol=2.0 ** -8, atol=1e-4)


def test_refusals():
    import torch

    import sparse_convolution_gb300 as fvx

    x = torch.zeros(4, 32, device="cuda")
    y, mean, rstd = fvx.layer_norm(x)
    w = torch.ones(31, device="cuda")
    for call in (lambda: fvx.layer_norm(x, w), lambda: fvx.layer_norm(x.double()), lambda: fvx.layer_norm(x.cpu()),
                 lambda: fvx.layer_norm(x, eps=-1.0), lambda: fvx.layer_norm(x, checkpoint_group=48),
                 lambda: fvx.layer_norm(x[0]), lambda: fvx.layer_norm(torch.zeros(2, 65537, device="cuda")),
                 lambda: fvx.layer_norm_backward(y[:3], x, mean, rstd),
                 lambda: fvx.layer_norm_backward(y, x, mean[:3], rstd),
                 lambda: fvx.layer_norm_backward(y.bfloat16(), x, mean, rstd),
                 lambda: fvx.Checkpoint8.pack(x, group=16),
                 lambda: fvx.Checkpoint8.pack(x).layer_norm(mean, rstd[:1])):
        with pytest.raises(fvx.FvxError) as e:
            call()
        assert e.value.status == "FVX_ERR_INVALID_ARG"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,pad", [(200_016, 64, 8), (200_000, 64, 16), (60_001, 256, 8), (300_009, 48, 8), (40_000, 1000, 24)])
def test_long_rows_apart(n, c, pad, dtype):
    """Rows a little apart, copied with what lies between them: the same bits as
    from dense ones, whatever lies there, and the last row's end is the tensor's."""
    import torch

    import sparse_convolution_gb300 as fvx

    x, w, b, dy = _inputs(n, c, dtype, 5 + pad)

    def apart(t):
        wide = torch.full((n * (c + pad) - pad,), float("nan"), dtype=t.dtype, device="cuda")
        view = wide.as_strided((n, c), (c + pad, 1))
        view.copy_(t)
        return view

    want = fvx.layer_norm(x, w, b, checkpoint_group=64)
    got = fvx.layer_norm(apart(x), w, b, checkpoint_group=64)
    assert all(torch.equal(p, q) for p, q in zip(want[:3], got[:3]))
    assert torch.equal(want[3].codes, got[3].codes) and torch.equal(want[3].steps, got[3].steps)
    packed = fvx.Checkpoint8.pack(apart(x), group=64)
    assert torch.equal(packed.codes, want[3].codes)
    for source, other in ((x, apart(x)), (want[3], want[3])):
        a = fvx.layer_norm_backward(dy, source, want[1], want[2], w)
        o = fvx.layer_norm_backward(apart(dy), other, want[1], want[2], w)
        assert torch.equal(a[0], o[0])
        # other stages, so the sums over the rows take another order: n terms of fp32
        for p, q in zip(a[1:], o[1:]):
            assert (p - q).abs().max() <= 2 * n * U * dy.float().abs().max() * 8
    fvx.device_status()
