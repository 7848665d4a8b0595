"""rotate_heads and norm_rotate_heads, forward and backward, against their
formulas in 64 bits at angles taken exactly from the Rotary's integer steps.

Tolerances.  u = 2^-24.  Sine and cosine: the fraction of a turn is cut at
2^-32 (1.5e-9 rad); its fp32 value and the two factors to radians make 3 u of at
most pi / 4; five or six rounded steps of the series 2 u; the magnitude's two
roundings 2 u: 8 u of the magnitude m in all.  A turned value u c - v s adds two
roundings: 12 u m (|u| + |v|).
Norm: sums of at most 32 positive products in a lane and 5 steps across lanes
make 40 u of the sum, 20 u of its root's reciprocal, whose instruction adds 4 u;
two products: 30 u of the value, with the rotation 48 u m (|a| + |b|).
Backward: with G = m (|dy_u| + |dy_v|) >= |g| and terms t = G |w x|,
  dx = rstd g w - x rstd^3 sum(g w x) / d:  100 u (rstd G |w| + |x| rstd^3 sum(t) / d),
  12 u of g, 30 u of rstd three times over, 40 u of the sum, 4 u of the products;
  dw: 42 u of each term G |x| rstd and fewer than 400 additions of it.
bf16 results add half a step, 2^-8 of the value (BF16_OUT_REL).
"""
import numpy as np
import pytest

from tests.gpu_common import BF16_OUT_REL

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, bound, what):
    err = np.abs(_np(got) - want)
    assert np.all(err <= bound), (what, float((err - bound).max()), float(err.max()))


def _angles(rotary, positions):
    """[tokens, pairs] radians: the steps' integers times the position, modulo 2^64, as a fraction of a turn."""
    pairs = rotary.size // 2
    axis = np.repeat(np.arange(rotary.axes), [pairs // rotary.axes + (a < pairs % rotary.axes) for a in range(rotary.axes)])
    at = positions.cpu().numpy().astype(np.int64).reshape(len(positions), rotary.axes)[:, axis].astype(np.uint64)  # two's complement
    with np.errstate(over="ignore"):
        part = (at * rotary.turns[None]).astype(np.int64)  # -half .. half a turn
    return part.astype(np.float64) / 2.0 ** 64 * (2 * np.pi)


def _places(rotary):
    p = np.arange(rotary.size // 2)
    return (p, p + rotary.size // 2) if rotary.layout == "half" else (2 * p, 2 * p + 1)


def _turn(x, rotary, angle, back=False):
    """(turned, m (|u| + |v|) at every channel; passing ones: themselves)"""
    if rotary is None:
        return x, np.abs(x)
    a, b = _places(rotary)
    m, c, s = float(rotary.magnitude), np.cos(angle)[:, None], np.sin(angle)[:, None] * (-1 if back else 1)
    y, size = x.copy(), np.abs(x)
    u, v = x[..., a], x[..., b]
    y[..., a], y[..., b] = m * (u * c - v * s), m * (v * c + u * s)
    size[..., a] = size[..., b] = m * (np.abs(u) + np.abs(v))
    return y, size


def _unit(x, eps):
    return 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def _rel(dtype):
    return BF16_OUT_REL if dtype == "bf16" else 0.0


def _check_rotate(got, x, rotary, angle, dtype, back=False):
    y, size = _turn(_np(x), rotary, angle, back)
    _close(got, y, 12 * U * size + _rel(dtype) * np.abs(y), "turned")


def _check_norm(got, x, w, rotary, angle, eps, dtype):
    xr = _np(x)
    y, size = _turn(xr * _unit(xr, eps) * w, rotary, angle)
    _close(got, y, 48 * U * size + _rel(dtype) * np.abs(y), "normed and turned")


def _check_norm_backward(dx, dw, dy, x, w, rotary, angle, eps, dtype):
    xr, d = _np(x), x.shape[2]
    rstd = _unit(xr, eps)
    g, size = _turn(_np(dy), rotary, angle, back=True)
    want = rstd * g * w - xr * rstd ** 3 * (g * w * xr).sum(-1, keepdims=True) / d
    bound = 100 * U * (rstd * size * np.abs(w) + np.abs(xr) * rstd ** 3 * (size * np.abs(w * xr)).sum(-1, keepdims=True) / d)
    _close(dx, want, bound + _rel(dtype) * np.abs(want), "dx")
    _close(dw, (g * xr * rstd).sum((0, 1)), (442 * U * size * np.abs(xr) * rstd).sum((0, 1)), "dweight")


def _heads(n, h, d, dtype, rng, pad=0, lead=0, extra=0):
    """[n, h, d] inside [n, h + extra, lead + d + pad]"""
    base = torch.zeros(n, h + extra, lead + d + pad, dtype=DT[dtype], device="cuda")
    x = base[:, :h, lead:lead + d]
    x.copy_(torch.from_numpy(rng.normal(size=(n, h, d)) * np.exp(0.5 * rng.normal(size=d)) + 0.1))
    return x


def _positions(n, axes, rng, span=1 << 31):
    at = rng.integers(-span, span, size=(n, axes))
    if n > 2 and span == 1 << 31:
        at[0], at[1], at[2] = -span, span - 1, 0
    return torch.from_numpy(at.astype(np.int32)).cuda()[:, 0] if axes == 1 else torch.from_numpy(at.astype(np.int32)).cuda()


# tokens, heads, key heads, size, rotated, axes, layout, padding, leading values: one token; sizes of one and of odd
# numbers; halves, bases and strides that allow 16-, 8-, 4- and 2-byte vectors; parts of the head; several items per lane
SHAPES = [(1, 16, 4, 128, 128, 1, "half", 0, 0), (1, 1, 0, 2, 2, 1, "interleaved", 0, 0), (5, 3, 1, 7, 4, 1, "interleaved", 0, 0),
          (70, 4, 2, 40, 40, 1, "half", 0, 0), (70, 4, 2, 40, 24, 2, "half", 0, 0), (33, 6, 3, 100, 60, 1, "interleaved", 3, 0),
          (257, 8, 8, 64, 64, 3, "half", 0, 0), (257, 8, 8, 64, 64, 3, "half", 8, 8), (130, 5, 0, 64, 64, 3, "interleaved", 4, 4),
          (50, 2, 2, 256, 256, 1, "half", 0, 0), (40, 1, 1, 256, 10, 1, "half", 0, 0), (40, 1, 1, 256, 64, 2, "interleaved", 1, 1),
          (19, 3, 1, 255, 254, 1, "half", 0, 0), (19, 3, 1, 254, 130, 3, "interleaved", 0, 0), (64, 5, 1, 80, 48, 2, "half", 2, 2),
          (1000, 2, 2, 16, 16, 3, "half", 0, 0), (9, 12, 1, 128, 2, 1, "half", 0, 0), (9, 12, 1, 129, 126, 1, "interleaved", 0, 0),
          (3001, 7, 2, 96, 96, 1, "interleaved", 0, 0), (20000, 8, 2, 64, 32, 3, "half", 0, 0), (4, 70, 1, 24, 4, 2, "half", 0, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,h,hk,d,rot,axes,layout,pad,lead", SHAPES)
def test_forward_and_backward(n, h, hk, d, rot, axes, layout, pad, lead, dtype):
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(n * 7919 + d * 31 + rot)
    rotary = fvx.Rotary(rot, axes=axes, layout=layout, base=700.0)
    at = _positions(n, axes, rng)
    angle = _angles(rotary, at)
    q, k = _heads(n, h, d, dtype, rng, pad, lead), _heads(n, hk, d, dtype, rng, pad, lead) if hk else None
    dq, dk = _heads(n, h, d, dtype, rng, pad), _heads(n, hk, d, dtype, rng) if hk else None
    wq, wk = (torch.from_numpy(1 + 0.3 * rng.normal(size=d)).float().cuda() for _ in range(2))
    both = lambda r: r if hk else (r, None)  # noqa: E731

    a, b = both(fvx.rotate_heads(q, at, rotary, k=k))
    _check_rotate(a, q, rotary, angle, dtype)
    ga, gb = both(fvx.rotate_heads_backward(dq, at, rotary, dk=dk))
    _check_rotate(ga, dq, rotary, angle, dtype, back=True)
    if hk:
        _check_rotate(b, k, rotary, angle, dtype)
        _check_rotate(gb, dk, rotary, angle, dtype, back=True)

    eps = 1e-5
    a, b = both(fvx.norm_rotate_heads(q, at, rotary, wq, k=k, k_weight=wk if hk else None, eps=eps))
    _check_norm(a, q, _np(wq), rotary, angle, eps, dtype)
    call = lambda: fvx.norm_rotate_heads_backward(dq, q, at, rotary, wq, dk=dk, k=k, k_weight=wk if hk else None,  # noqa: E731
                                                  eps=eps)
    got = call()
    _check_norm_backward(got[0], got[2 if hk else 1], dq, q, _np(wq), rotary, angle, eps, dtype)
    if hk:
        _check_norm(b, k, _np(wk), rotary, angle, eps, dtype)
        _check_norm_backward(got[1], got[3], dk, k, _np(wk), rotary, angle, eps, dtype)
    assert all(torch.equal(x, y) for x, y in zip(got, call()))  # the sums' order is fixed
    fvx.device_status()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,h,d,pad", [(300, 4, 64, 0), (31, 2, 1, 0), (31, 2, 3, 2), (12, 1, 256, 0), (50, 3, 77, 0)])
def test_norm_without_rotation_and_weight(n, h, d, pad, dtype):
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(n + d)
    x, dy = _heads(n, h, d, dtype, rng, pad), _heads(n, h, d, dtype, rng)
    one = np.ones(d)
    _check_norm(fvx.norm_rotate_heads(x, eps=1e-6), x, one, None, None, 1e-6, dtype)
    dx, dw = fvx.norm_rotate_heads_backward(dy, x, eps=1e-6)
    _check_norm_backward(dx, dw, dy, x, one, None, None, 1e-6, dtype)


def test_tensors_of_their_own_tokens():
    """Queries and keys of different numbers, positions and weights (one without) in one launch."""
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(1)
    rotary = fvx.Rotary(48, axes=2, layout="interleaved")
    q, k = _heads(77, 4, 64, "bf16", rng), _heads(1300, 2, 64, "bf16", rng)
    aq, ak = _positions(77, 2, rng), _positions(1300, 3, rng)[:, 1:]  # a part of wider rows
    w = torch.from_numpy(rng.normal(size=64)).float().cuda()
    a, b = fvx.norm_rotate_heads(q, aq, rotary, None, k=k, k_positions=ak, k_weight=w)
    _check_norm(a, q, np.ones(64), rotary, _angles(rotary, aq), 1e-6, "bf16")
    _check_norm(b, k, _np(w), rotary, _angles(rotary, ak), 1e-6, "bf16")
    dq, dk = _heads(77, 4, 64, "bf16", rng), _heads(1300, 2, 64, "bf16", rng)
    gq, gk, dw, dwk = fvx.norm_rotate_heads_backward(dq, q, aq, rotary, None, dk=dk, k=k, k_positions=ak, k_weight=w)
    _check_norm_backward(gq, dw, dq, q, np.ones(64), rotary, _angles(rotary, aq), 1e-6, "bf16")
    _check_norm_backward(gk, dwk, dk, k, _np(w), rotary, _angles(rotary, ak), 1e-6, "bf16")


@pytest.mark.parametrize("nq,nk", [(0, 0), (0, 9), (9, 0)])
def test_no_tokens(nq, nk):
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(2)
    rotary = fvx.Rotary(16)
    q, k = _heads(nq, 2, 16, "f32", rng), _heads(nk, 3, 16, "f32", rng)
    aq, ak = _positions(nq, 1, rng), _positions(nk, 1, rng)
    a, b = fvx.rotate_heads(q, aq, rotary, k=k, k_positions=ak)
    _check_rotate(a, q, rotary, _angles(rotary, aq), "f32")
    _check_rotate(b, k, rotary, _angles(rotary, ak), "f32")
    gq, gk, dw, dwk = fvx.norm_rotate_heads_backward(q, q, aq, rotary, dk=k, k=k, k_positions=ak)
    assert gq.shape == q.shape and gk.shape == k.shape
    one = np.ones(16)
    _check_norm_backward(gq, dw, q, q, one, rotary, _angles(rotary, aq), 1e-6, "f32")
    _check_norm_backward(gk, dwk, k, k, one, rotary, _angles(rotary, ak), 1e-6, "f32")


def test_no_tokens_of_repeated_heads():
    """An empty result has whatever strides its tensor had: nothing lies over anything."""
    import sparse_convolution_gb300 as fvx

    q = torch.empty(0, 1, 16, device="cuda").expand(0, 5, 16)
    assert fvx.norm_rotate_heads(q).shape == (0, 5, 16)


@pytest.mark.parametrize("scaling", ["linear", "base", "parts"])
def test_stretched_contexts(scaling):
    """The steps themselves are tested on the host; here the magnitude and far positions, exactly in turns."""
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(4)
    rotary = fvx.Rotary(96, scaling=scaling, factor=16.0, length=8192 if scaling == "parts" else None)
    q, at = _heads(400, 2, 128, "f32", rng), _positions(400, 1, rng, 1 << 20)
    angle = _angles(rotary, at)
    _check_rotate(fvx.rotate_heads(q, at, rotary), q, rotary, angle, "f32")
    _check_rotate(fvx.rotate_heads_backward(q, at, rotary), q, rotary, angle, "f32", back=True)
    dx, dw = fvx.norm_rotate_heads_backward(q, q, at, rotary)
    _check_norm_backward(dx, dw, q, q, np.ones(128), rotary, angle, 1e-6, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_position_zero_changes_nothing(dtype):
    import sparse_convolution_gb300 as fvx

    q = _heads(40, 3, 64, dtype, np.random.default_rng(5))
    at = torch.zeros(40, dtype=torch.int32, device="cuda")
    assert torch.equal(fvx.rotate_heads(q, at, fvx.Rotary(64)), q)


def test_gradients_against_differences():
    """Central differences of the definition in 64 bits along random directions: h = 1e-4 leaves a truncation of
    about h^2 and a rounding of about 1e-16 / h, both far below the fp32 gradient's own error (100 u of the terms'
    sizes: 6e-6)."""
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(6)
    rotary = fvx.Rotary(20, axes=2, layout="interleaved")
    x, dy, at = _heads(21, 3, 26, "f32", rng), _heads(21, 3, 26, "f32", rng), _positions(21, 2, rng)
    w = torch.from_numpy(1 + 0.3 * rng.normal(size=26)).float().cuda()
    dx, dw = (_np(t) for t in fvx.norm_rotate_heads_backward(dy, x, at, rotary, w, eps=1e-3))
    X, W, D, angle = _np(x), _np(w), _np(dy), _angles(rotary, at)
    f = lambda x_, w_: float((_turn(x_ * _unit(x_, 1e-3) * w_, rotary, angle)[0] * D).sum())  # noqa: E731
    h = 1e-4
    for _ in range(4):
        ux, uw = rng.normal(size=X.shape), rng.normal(size=26)
        num = (f(X + h * ux, W + h * uw) - f(X - h * ux, W - h * uw)) / (2 * h)
        size = np.abs(dx * ux).sum() + np.abs(dw * uw).sum()
        assert abs(num - (dx * ux).sum() - (dw * uw).sum()) <= 1e-5 * size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_in_one_products_rows(layout, dtype):
    """Queries and keys are turned where they lie, between the values and whatever else their rows hold."""
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(7)
    rotary, at = fvx.Rotary(32, axes=3, layout=layout), _positions(900, 3, rng, 4000)
    qkv = torch.from_numpy(rng.normal(size=(900, 4 + 2 + 2, 64))).cuda().to(DT[dtype])
    before = qkv.clone()
    q, k = qkv[:, :4], qkv[:, 4:6]
    want = fvx.norm_rotate_heads(q, at, rotary, k=k)
    got = fvx.norm_rotate_heads(q, at, rotary, k=k, out=(q, k))
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, 6:], before[:, 6:])
    # the gradient in the result's place, and in the input's
    dy, x = before[:, :4].clone(), before[:, 4:].clone()
    dx, _ = fvx.norm_rotate_heads_backward(dy, x, at, rotary)
    for place in ("dy", "x"):
        a, b = dy.clone(), x.clone()
        fvx.norm_rotate_heads_backward(a, b, at, rotary, out=a if place == "dy" else b)
        assert torch.equal(a if place == "dy" else b, dx)


def test_strided_and_repeated_inputs():
    """A last dimension with gaps, tokens that are all the same row, heads in another order of memory."""
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(8)
    rotary, at = fvx.Rotary(24), _positions(50, 1, rng)
    base = _heads(50, 4, 64, "f32", rng)
    for q in (base[:, :, ::2], base[:1].expand(50, 4, 64), base.permute(1, 0, 2).contiguous().permute(1, 0, 2),
              base[:, :1].expand(50, 6, 64)):
        _check_rotate(fvx.rotate_heads(q, at, rotary), q, rotary, _angles(rotary, at), "f32")
        dx, dw = fvx.norm_rotate_heads_backward(q, q, at, rotary)
        _check_norm_backward(dx, dw, q, q, np.ones(q.shape[2]), rotary, _angles(rotary, at), 1e-6, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_not_finite_stays_where_it_is(dtype):
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(9)
    rotary, at = fvx.Rotary(16), _positions(64, 1, rng)
    q = _heads(64, 4, 40, dtype, rng)
    clean = fvx.rotate_heads(q, at, rotary), fvx.norm_rotate_heads(q, at, rotary), \
        fvx.norm_rotate_heads_backward(q, q, at, rotary)[0]
    q[5, 2, 30] = float("inf")   # a value that passes
    q[6, 1, 3] = float("nan")    # paired with 11
    got = fvx.rotate_heads(q, at, rotary)
    same = got == clean[0]
    assert torch.isinf(got[5, 2, 30]) and torch.isnan(got[6, 1, [3, 11]]).all()
    assert int((~same).sum()) == 3
    for got, want in zip((fvx.norm_rotate_heads(q, at, rotary), fvx.norm_rotate_heads_backward(q, q, at, rotary)[0]),
                         clean[1:]):
        same = (got == want).all(2)
        same[5, 2] = same[6, 1] = True
        assert same.all()


def test_heads_of_zeros():
    """1 / sqrt(eps) times nothing: zeros, and the gradient's plain product."""
    import sparse_convolution_gb300 as fvx

    x = torch.zeros(3, 2, 32, device="cuda")
    dy = torch.ones_like(x)
    assert not fvx.norm_rotate_heads(x, eps=1e-6).any()
    dx, dw = fvx.norm_rotate_heads_backward(dy, x, eps=1e-6)
    assert torch.allclose(dx, torch.full_like(dx, 1e3), rtol=1e-6) and not dw.any()


def test_offsets_past_32_bits():
    """Tokens 2^31 + 64 values apart."""
    import sparse_convolution_gb300 as fvx

    step = (1 << 31) + 64
    store = torch.empty(2 * step + 4 * 64, dtype=torch.bfloat16, device="cuda")
    q = store.as_strided((3, 4, 64), (step, 64, 1))
    rng = np.random.default_rng(10)
    q.copy_(torch.from_numpy(rng.normal(size=(3, 4, 64))))
    rotary, at = fvx.Rotary(64), _positions(3, 1, rng)
    want = fvx.norm_rotate_heads(q.contiguous(), at, rotary)
    assert torch.equal(fvx.norm_rotate_heads(q, at, rotary), want)
    assert torch.equal(fvx.norm_rotate_heads(q, at, rotary, out=q), want) and torch.equal(q, want)


def test_on_another_stream_and_captured():
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(11)
    rotary, at = fvx.Rotary(64, axes=3), _positions(5000, 3, rng, 500)
    q, k, dq, dk = (_heads(5000, h, 64, "bf16", rng) for h in (8, 2, 8, 2))
    w = torch.ones(64, device="cuda")

    def step():
        a = fvx.norm_rotate_heads(q, at, rotary, w, k=k, k_weight=w)
        b = fvx.norm_rotate_heads_backward(dq, q, at, rotary, w, dk=dk, k=k, k_weight=w)
        return [*a, *b, fvx.rotate_heads(q, at, rotary)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fvx.norm_rotate_heads(q, at, rotary, w, k=k, k_weight=w, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    # two graphs, replayed in turn: neither reads what the other left
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        held2 = step()
    for t in (q, k, dq, dk):
        t.mul_(-1.5)
    want = step()
    for g in (graph, other, graph):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, want)) and all(torch.equal(x, y) for x, y in zip(held2, want))


def test_refusals():
    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(12)
    q, k, at, r = _heads(6, 2, 16, "f32", rng), _heads(6, 1, 16, "f32", rng), _positions(6, 1, rng), fvx.Rotary(16)
    w = torch.ones(16, device="cuda")
    f, g, b = fvx.rotate_heads, fvx.norm_rotate_heads, fvx.norm_rotate_heads_backward
    for call in (lambda: f(q.half(), at, r), lambda: f(q[0], at, r), lambda: f(q, at.long(), r), lambda: f(q, at[:5], r),
                 lambda: f(q, at.float(), r), lambda: f(q, at.cpu(), r), lambda: f(q.cpu(), at, r), lambda: f(q, None, r),
                 lambda: f(q, at, None), lambda: f(q, at, fvx.Rotary(16, axes=2)), lambda: f(q, at, fvx.Rotary(18)),
                 lambda: f(q, at, r, k=k.bfloat16()), lambda: f(q, at, r, k=k[:, :, :8]), lambda: f(q, at, r, k=k[:3]),
                 lambda: f(q, at, r, k_positions=at), lambda: f(q, at, r, out=(q, k)), lambda: f(q, at, r, k=k, out=q),
                 lambda: f(q, at, r, out=q[:, :, :8]), lambda: f(q, at, r, out=q.bfloat16()),
                 lambda: f(q, at, r, out=q[:1].expand(6, 2, 16)), lambda: f(q[:, :0], at, r),
                 lambda: g(q, at, r, w[:8]), lambda: g(q, at, r, w.double()),
                 lambda: g(q, at, r, k_weight=w), lambda: g(q, at, r, eps=-1.0), lambda: g(q, None, r),
                 lambda: b(k, q, at, r), lambda: b(q.bfloat16(), q, at, r), lambda: b(q, q, at, r, k=k),
                 lambda: b(q, q, at, r, dk=k), lambda: b(q, q, at, r, dk=q, k=k), lambda: g(torch.zeros(2, 1, 257, device="cuda"))):
        with pytest.raises(fvx.FvxError) as e:
            call()
        assert e.value.status == "FVX_ERR_INVALID_ARG"


def test_calls_at_once():
    """Host threads on streams of their own, whose calls take different kernels and amounts of shared memory."""
    import threading

    import sparse_convolution_gb300 as fvx

    rng = np.random.default_rng(13)
    calls = []
    for n, h, d, dtype in ((20000, 8, 64, "bf16"), (7000, 6, 80, "bf16"), (9000, 4, 40, "f32"), (3, 2, 128, "bf16")):
        q, dq = _heads(n, h, d, dtype, rng), _heads(n, h, d, dtype, rng)
        at, rotary, w = _positions(n, 3, rng), fvx.Rotary(d // 4 * 2, axes=3), torch.ones(d, device="cuda")

        def call(q=q, dq=dq, at=at, rotary=rotary, w=w):
            return [fvx.norm_rotate_heads(q, at, rotary, w), *fvx.norm_rotate_heads_backward(dq, q, at, rotary, w),
                    fvx.dropout(q, 0.3, 5, 6, residual=dq)]

        calls.append((call, call()))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(calls))

    def work(call, want):
        side = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(side):
            for _ in range(30):
                got = call()
            side.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                failed.append(want[0].shape)

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    fvx.device_status()
    assert not failed, failed
