"""Cross attention of ragged batches, forward and backward, against a plain
implementation in 64 bits.

Tolerances.  u = 2^-24; a score is within e_s = (size + 3) u scale sum|q||k| of
the exact one, a probability within a relative 2 e_s + 8 u of it, and a sum of
m terms within m u sum|terms|.  bf16 adds the rounding of the stored results
(BF16_OUT_REL of the value), of the probabilities and of the score gradients that
enter the products (as much of each), and of `out`, which the backward pass reads
(as much of sum|dout||out| in delta).
"""
import numpy as np
import pytest

from tests.gpu_common import BF16_OUT_REL

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": "float32", "bf16": "bfloat16"}


def _offs(lens):
    return [0] + [int(v) for v in np.cumsum(lens)]


def _case(qlens, klens, heads, kv_heads, d, dtype, seed, drop=0.0, sharp=1.0):
    import torch

    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(getattr(torch, DT[dtype])).cuda()  # noqa: E731
    nq, nk = sum(qlens), sum(klens)
    t = {"q": r(nq, heads, d) * sharp, "k": r(nk, kv_heads, d), "v": r(nk, kv_heads, d), "dout": r(nq, heads, d)}
    mask = None
    if drop:
        mask = (torch.rand(nk, generator=g) >= drop).cuda()
    return t, _offs(qlens), _offs(klens), mask


def _np(t):
    return t.detach().double().cpu().numpy()


def _reference(t, qo, ko, mask, scale, backward=True):
    """Values and error bounds, sample by sample and head by head."""
    q, k, v, do = (_np(t[n]) for n in ("q", "k", "v", "dout"))
    heads, kv_heads, d = q.shape[1], k.shape[1], q.shape[2]
    keep_all = np.ones(k.shape[0], bool) if mask is None else mask.cpu().numpy().astype(bool)
    bf = t["q"].dtype.itemsize == 2
    rr = BF16_OUT_REL if bf else 0.0
    out, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    z = lambda a: np.zeros_like(a)  # noqa: E731
    ref = dict(out=out, lse=lse, dq=z(q), dk=z(k), dv=z(v))
    bound = {n: z(a) for n, a in ref.items()}
    for b in range(len(qo) - 1):
        qs = slice(qo[b], qo[b + 1])
        ks = np.arange(ko[b], ko[b + 1])[keep_all[ko[b]:ko[b + 1]]]
        if qs.start == qs.stop or not len(ks):
            continue
        for h in range(heads):
            kh = h // (heads // kv_heads)
            Q, K, V, D = q[qs, h], k[ks, kh], v[ks, kh], do[qs, h]
            s = Q @ K.T * scale
            es = ((d + 3) * U * abs(scale) * (np.abs(Q) @ np.abs(K).T)).max(1, keepdims=True)
            top = s.max(1, keepdims=True)
            ex = np.exp(s - top)
            tot = ex.sum(1, keepdims=True)
            p = ex / tot
            m = len(ks) + 64
            ep = 2 * es + (8 + m) * U  # relative error of a normalised probability
            o = p @ V
            out[qs, h] = o
            lse[qs, h] = (top + np.log(tot))[:, 0]
            bound["lse"][qs, h] = (es + (8 + m) * U + 4 * U * np.abs(top + np.log(tot)))[:, 0]
            bo = (ep + rr + m * U) * (p @ np.abs(V)) + rr * np.abs(o)
            bound["out"][qs, h] = bo
            if not backward:
                continue
            dp = D @ V.T
            delta = (D * o).sum(1, keepdims=True)
            edelta = (np.abs(D) * bo).sum(1, keepdims=True) + d * U * (np.abs(D) * np.abs(o)).sum(1, keepdims=True)
            edp = d * U * (np.abs(D) @ np.abs(V).T)
            ds = p * (dp - delta) * scale
            eds = abs(scale) * p * ((edp + edelta) + (ep + 4 * U) * np.abs(dp - delta)) + rr * np.abs(ds)
            n = Q.shape[0] * (heads // kv_heads) + 64
            dq, dk, dv = ds @ K, ds.T @ Q, p.T @ D
            ref["dq"][qs, h] = dq
            ref["dk"][ks, kh] += dk
            ref["dv"][ks, kh] += dv
            bound["dq"][qs, h] = eds @ np.abs(K) + m * U * (np.abs(ds) @ np.abs(K)) + rr * np.abs(dq)
            bound["dk"][ks, kh] += eds.T @ np.abs(Q) + n * U * (np.abs(ds).T @ np.abs(Q)) + rr * np.abs(dk)
            bound["dv"][ks, kh] += (p * (ep + rr)).T @ np.abs(D) + n * U * (p.T @ np.abs(D)) + rr * np.abs(dv)
    return ref, bound


def _close(got, want, bound, name):
    got = _np(got)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine]), name
    err = np.abs(got[fine] - want[fine])
    assert np.all(err <= bound[fine] * 1.01 + 1e-30), (name, float((err - bound[fine]).max()), float(err.max()))


def _run(t, qo, ko, mask, scale=None, stream=None, backward=True):
    import sparse_convolution_gb300 as fvx

    out, lse = fvx.cross_attention(t["q"], t["k"], t["v"], qo, ko, key_mask=mask, scale=scale, stream=stream)
    got = dict(out=out, lse=lse)
    if backward:
        got["dq"], got["dk"], got["dv"] = fvx.cross_attention_backward(t["dout"], t["q"], t["k"], t["v"], out, lse, qo,
                                                                       ko, key_mask=mask, scale=scale, stream=stream)
    return got


def _check(t, qo, ko, mask, scale=None, backward=True):
    import sparse_convolution_gb300 as fvx

    got = _run(t, qo, ko, mask, scale, backward=backward)
    fvx.device_status()
    ref, bound = _reference(t, qo, ko, mask, t["q"].shape[2] ** -0.5 if scale is None else scale, backward)
    for n in got:
        _close(got[n], ref[n], bound[n], n)
    return got


# lengths of zero and one, tiles that end at, before and after 64 and 128
# rows or keys, shared key heads (odd groups too), odd head sizes
CASES = [
    ([1], [1], 1, 1, 64), ([1, 1, 1], [300, 1, 129], 8, 2, 128), ([0, 5, 0], [7, 0, 3], 2, 1, 32), ([3], [0], 2, 2, 64),
    ([127, 128, 129], [64, 63, 65], 2, 2, 64), ([200, 1, 77], [128, 127, 129], 4, 1, 64), ([65, 260], [255, 257], 6, 2, 40),
    ([130], [500], 5, 1, 16), ([300], [33], 3, 3, 128), ([64, 64], [192, 320], 12, 4, 96), ([31, 500], [77, 12], 8, 8, 64),
    ([90], [400], 7, 1, 80), ([2, 600, 3], [1000, 130, 1], 4, 2, 128), ([257], [256], 10, 2, 72), ([40], [90], 3, 1, 8),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("qlens,klens,heads,kv_heads,d", CASES)
def test_forward_and_backward(qlens, klens, heads, kv_heads, d, drop, dtype):
    t, qo, ko, mask = _case(qlens, klens, heads, kv_heads, d, dtype, sum(qlens) * 7 + sum(klens) + d, drop)
    got = _check(t, qo, ko, mask)
    again = _run(t, qo, ko, mask)
    assert all((got[n] == again[n]).all() for n in got)  # the sums' order is fixed


@pytest.mark.parametrize("dtype,d", [("f32", 20), ("f32", 1), ("f32", 100), ("bf16", 20), ("bf16", 1), ("bf16", 100)])
def test_odd_head_sizes(dtype, d):
    t, qo, ko, mask = _case([70, 9], [66, 130], 4, 2, d, dtype, d, 0.2)
    _check(t, qo, ko, mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_keys_few_queries(dtype):
    """The keys are split over many units whose results are joined."""
    t, qo, ko, mask = _case([1, 3, 2], [5000, 9001, 17], 8, 2, 64, dtype, 3, 0.1)
    _check(t, qo, ko, mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("qlens,klens,heads,kv_heads,d", [
    ([1], [1], 1, 1, 8), ([1, 0, 1], [37, 5, 0], 8, 1, 64), ([1, 1], [129, 4000], 8, 2, 128), ([2, 3], [600, 31], 2, 2, 40),
    ([1], [70000], 4, 4, 32), ([1] * 40, [50 + 7 * i for i in range(40)], 6, 2, 96), ([8, 7], [1000, 3], 1, 1, 128),
    ([1, 1, 1], [255, 256, 257], 7, 1, 72)])
def test_a_few_rows(qlens, klens, heads, kv_heads, d, dtype):
    """At most eight rows per key head: lengths around a block's turn, many
    samples, one sample long enough for several clusters, none kept."""
    for drop in (0.0, 0.4):
        t, qo, ko, mask = _case(qlens, klens, heads, kv_heads, d, dtype, sum(klens) + d, drop)
        got = _check(t, qo, ko, mask, backward=False)
        again = _run(t, qo, ko, mask, backward=False)
        assert all((got[n] == again[n]).all() for n in got)


@pytest.mark.parametrize("drop", [0.0, 0.4])
@pytest.mark.parametrize("qlens,klens,heads,kv_heads,d", [
    ([16], [200], 2, 2, 40), ([5, 0, 1], [700, 3, 64], 6, 2, 100), ([4, 8], [65, 130], 4, 2, 128), ([9], [1], 3, 3, 20),
    ([10, 32, 1], [129, 0, 400], 2, 2, 64), ([8, 7], [513, 64], 12, 3, 128), ([17], [63], 1, 1, 12),
    ([200, 33, 0], [16, 1, 9], 4, 4, 40), ([300], [7], 6, 2, 128), ([64, 129], [15, 16], 2, 1, 100), ([16], [16], 2, 2, 32)])
def test_small_tiles(qlens, klens, heads, kv_heads, d, drop):
    """fp32 tiles of 16 and 32 rows, and of 16 keys."""
    _check(*_case(qlens, klens, heads, kv_heads, d, "f32", 61, drop=drop))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.5, -0.7, 0.0])
def test_a_few_rows_that_hold_anything(scale, dtype):
    """Masked keys of NaN and infinities, a sample of none but those, sharp,
    negative and no scores."""
    import torch

    t, qo, ko, _ = _case([1, 2, 1], [300, 40, 200], 4, 2, 64, dtype, 31)
    mask = torch.ones(ko[-1], dtype=torch.bool, device="cuda")
    mask[5:290:4] = False
    mask[ko[1]:ko[2]] = False
    clean = _check(t, qo, ko, mask, scale=scale, backward=False)
    t["k"][~mask], t["v"][~mask] = float("nan"), float("inf")
    got = _run(t, qo, ko, mask, scale=scale, backward=False)
    assert all(torch.equal(got[n], clean[n]) for n in got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_queries_few_keys(dtype):
    """The rows are split over many units whose key gradients are summed."""
    t, qo, ko, mask = _case([6000, 3001], [5, 70], 4, 4, 64, dtype, 4, 0.2)
    _check(t, qo, ko, mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_items(dtype):
    """More batch elements than the kernel arguments hold, empty ones among them."""
    rng = np.random.default_rng(0)
    ql, kl = rng.integers(0, 9, 700), rng.integers(0, 7, 700)
    t, qo, ko, mask = _case(ql.tolist(), kl.tolist(), 4, 2, 32, dtype, 5, 0.3)
    _check(t, qo, ko, mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", ["nan", "inf", "lowest"])
def test_masked_keys_hold_anything(bad, dtype):
    """What a masked key's row holds reaches nothing; a sample without kept
    keys gets zeros; neither do a neighbouring sample's rows."""
    import torch

    t, qo, ko, _ = _case([70, 33, 140], [150, 40, 129], 4, 2, 64, dtype, 6)
    mask = torch.ones(ko[-1], dtype=torch.bool, device="cuda")
    mask[3:60:3] = False
    mask[ko[1]:ko[2]] = False
    mask[ko[2]:ko[2] + 128] = False  # one kept key, in the second tile
    clean = _check(t, qo, ko, mask)
    fill = {"nan": float("nan"), "inf": float("inf"), "lowest": torch.finfo(t["k"].dtype).min}[bad]
    t["k"][~mask] = fill
    t["v"][~mask] = fill
    got = _run(t, qo, ko, mask)
    for n in got:
        assert torch.equal(got[n], clean[n]), n
    assert not got["out"][qo[1]:qo[2]].any() and torch.isneginf(got["lse"][qo[1]:qo[2]]).all()
    assert not got["dq"][qo[1]:qo[2]].any() and not got["dk"][~mask].any() and not got["dv"][~mask].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_neighbour_that_is_not_finite(dtype):
    """NaN in one sample's queries, keys and values leaves the samples beside it
    bit for bit, though tiles reach past a sample's end."""
    import torch

    t, qo, ko, _ = _case([70, 33, 140], [150, 40, 129], 4, 2, 64, dtype, 7)
    clean = _run(t, qo, ko, None)
    for n, o in (("q", qo), ("dout", qo), ("k", ko), ("v", ko)):
        t[n][o[1]:o[2]] = float("nan")
    got = _run(t, qo, ko, None)
    for n, o in (("out", qo), ("lse", qo), ("dq", qo), ("dk", ko), ("dv", ko)):
        for b in (0, 2):
            assert torch.equal(got[n][o[b]:o[b + 1]], clean[n][o[b]:o[b + 1]]), n
        assert torch.isnan(got[n][o[1]:o[2]].float()).all(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [3.0, -0.5, 0.0])
def test_scales(scale, dtype):
    """Sharp, negative and no scores: the running maximum moves by much."""
    t, qo, ko, mask = _case([100, 30], [300, 200], 4, 2, 64, dtype, 8)
    _check(t, qo, ko, mask, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rising_scores(dtype):
    """Keys that grow along the sample: every tile has a new, much larger maximum."""
    import torch

    t, qo, ko, mask = _case([140], [700], 2, 1, 64, dtype, 9)
    ramp = torch.linspace(0.0, 6.0, 700, device="cuda")[:, None, None]
    t["k"] = (t["k"] * ramp).to(t["k"].dtype)
    _check(t, qo, ko, mask)


@pytest.mark.parametrize("reach", [1.0, 4.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scores_far_from_zero(dtype, d, reach):
    """First tiles whose scores all lie far above or below 0, near the limits of
    what is taken relative to 0, and rows of each kind side by side; a later
    tile's scores on the other side."""
    import torch

    t, qo, ko, mask = _case([300], [400], 2, 2, d, dtype, 71)
    t["q"].mul_(0.05)
    t["k"].mul_(0.05)
    t["q"][:, :, 0] = torch.linspace(-12.0, 12.0, 300, device="cuda").to(t["q"].dtype)[:, None]
    # scores of about +-12 (48) in the first tile, half of that, turned round, in the last
    t["k"][:128, :, 0] = reach * d ** 0.5
    t["k"][128:, :, 0] = 0.0
    t["k"][384:, :, 0] = -0.5 * reach * d ** 0.5
    _check(t, qo, ko, mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layouts(dtype):
    """Tensors cut out of wider ones, heads before tokens, heads broadcast."""
    import torch

    t, qo, ko, mask = _case([50, 77], [140, 66], 4, 2, 64, dtype, 10, 0.2)
    want = _run(t, qo, ko, mask)
    views = {}
    for n, x in t.items():
        wide = torch.full((x.shape[0], x.shape[1] * 2 + 1, x.shape[2] + 8), float("nan"), device="cuda", dtype=x.dtype)
        wide[:, 1::2, :x.shape[2]] = x
        views[n] = wide[:, 1::2, :x.shape[2]]
    swapped = {n: x.transpose(0, 1).contiguous().transpose(0, 1) for n, x in t.items()}
    odd = {}
    for n, x in t.items():
        wide = torch.full((x.shape[0], x.shape[1], x.shape[2] + 3), float("nan"), device="cuda", dtype=x.dtype)
        wide[:, :, 1:-2] = x
        odd[n] = wide[:, :, 1:-2]
    for kind in (views, swapped, odd):
        got = _run(kind, qo, ko, mask)
        for n in got:
            assert torch.equal(got[n], want[n]), n
    one = dict(t, k=t["k"][:, :1].expand(-1, 2, -1), v=t["v"][:, :1].expand(-1, 2, -1))
    _check(one, qo, ko, mask)


def test_gradients_against_differences():
    """Central differences of the definition in 64 bits along random directions
    (h = 1e-4: truncation about h^2, rounding about 1e-16 / h)."""
    t, qo, ko, mask = _case([13, 9], [21, 34], 4, 2, 24, "f32", 12, 0.2)
    got = {n: _np(x) for n, x in _run(t, qo, ko, mask).items()}
    base = {n: _np(x) for n, x in t.items()}
    keep = mask.cpu().numpy()

    def f(q, k, v):
        total = 0.0
        for b in range(2):
            at = np.arange(ko[b], ko[b + 1])[keep[ko[b]:ko[b + 1]]]
            for h in range(4):
                s = q[qo[b]:qo[b + 1], h] @ k[at, h // 2].T * 24 ** -0.5
                p = np.exp(s - s.max(1, keepdims=True))
                total += ((p / p.sum(1, keepdims=True)) @ v[at, h // 2] * base["dout"][qo[b]:qo[b + 1], h]).sum()
        return total

    rng = np.random.default_rng(1)
    h = 1e-4
    for _ in range(4):
        u = {n: rng.normal(size=base[n].shape) for n in "qkv"}
        num = (f(*(base[n] + h * u[n] for n in "qkv")) - f(*(base[n] - h * u[n] for n in "qkv"))) / (2 * h)
        parts = [got["d" + n] * u[n] for n in "qkv"]
        assert abs(num - sum(p.sum() for p in parts)) <= 2e-5 * sum(np.abs(p).sum() for p in parts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_another_stream(dtype):
    import torch

    t, qo, ko, mask = _case([500, 900], [200, 333], 4, 2, 64, dtype, 13, 0.1)
    want = _run(t, qo, ko, mask)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _run(t, qo, ko, mask, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for n in got:
        assert torch.equal(got[n], want[n]), n


def test_captured_in_a_graph():
    """Both passes recorded once and replayed on new values."""
    import torch

    import sparse_convolution_gb300 as fvx

    t, qo, ko, mask = _case([200, 90], [130, 257], 4, 2, 64, "bf16", 14, 0.1)
    _run(t, qo, ko, mask)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(t, qo, ko, mask)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _run(t, qo, ko, mask)
    t2, _, _, _ = _case([200, 90], [130, 257], 4, 2, 64, "bf16", 15)
    for n in t:
        t[n].copy_(t2[n])
    g.replay()
    want = _run(t, qo, ko, mask)
    for n in got:
        assert torch.equal(got[n], want[n]), n
    fvx.device_status()


def test_long_cache_offsets():
    """Keys and values of more than 2^31 elements: the last sample's are found."""
    import torch

    import sparse_convolution_gb300 as fvx

    heads, d = 16, 128
    far = (1 << 31) // (heads * d) + 5
    t, _, _, _ = _case([3], [200], heads, heads, d, "bf16", 16)
    k = torch.zeros(far + 200, heads, d, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    k[far:], v[far:] = t["k"], t["v"]
    out, lse = fvx.cross_attention(t["q"], k, v, [0, 0, 3], [0, far, far + 200])
    want, lwant = fvx.cross_attention(t["q"], t["k"], t["v"], [0, 3], [0, 200])
    assert torch.equal(out, want) and torch.equal(lse, lwant)


def test_refusals():
    import torch

    import sparse_convolution_gb300 as fvx

    t, qo, ko, _ = _case([5], [7], 4, 2, 16, "f32", 0)
    q, k, v = t["q"], t["k"], t["v"]
    out, lse = fvx.cross_attention(q, k, v, qo, ko)
    big = torch.zeros(5, 4, 129, device="cuda")
    for call in (lambda: fvx.cross_attention(q, k, v, [0, 4], ko), lambda: fvx.cross_attention(q, k, v, [0, 5], [0, 3, 7]),
                 lambda: fvx.cross_attention(q, k, v, [0, 6, 5], [0, 7, 7]),
                 lambda: fvx.cross_attention(q, k, v, [1, 5], ko),
                 lambda: fvx.cross_attention(q, k.bfloat16(), v, qo, ko),
                 lambda: fvx.cross_attention(q[:, :3], k, v, qo, ko), lambda: fvx.cross_attention(q, k, v[:6], qo, ko),
                 lambda: fvx.cross_attention(big, big, big, qo, [0, 5]),
                 lambda: fvx.cross_attention(q.cpu(), k, v, qo, ko),
                 lambda: fvx.cross_attention(q, k, v, qo, ko, key_mask=torch.ones(6, dtype=torch.bool, device="cuda")),
                 lambda: fvx.cross_attention(q, k, v, qo, ko, scale=float("nan")),
                 lambda: fvx.cross_attention_backward(t["dout"][:4], q, k, v, out, lse, qo, ko),
                 lambda: fvx.cross_attention_backward(t["dout"], q, k, v, out, lse[:4], qo, ko)):
        with pytest.raises(fvx.FvxError) as e:
            call()
        assert e.value.status == "FVX_ERR_INVALID_ARG"
