"""Rotary steps against their definition, Philox against its published vectors,
and the refusals of the head and dropout entry points: all on the host, before
any CUDA work (no GPU needed)."""
import ctypes
import math
import struct

import numpy as np
import pytest

from tests.helpers_dropout import philox

INVALID, RANGE, OK = 1, 2, 0
P = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from sparse_convolution_gb300 import build_lib

    build_lib.build()
    import sparse_convolution_gb300 as fvx

    return fvx.load()


# ---------------------------------------------------------------- rotary steps
def _frequencies(pairs, base, scaling, factor, length):
    out = []
    for n in pairs:
        for i in range(n):
            b = base * factor ** (n / (n - 1)) if scaling == "base" and n > 1 else base
            f = b ** (-i / n)
            if scaling == "linear":
                f /= factor
            if scaling == "parts":
                keep = min(1.0, max(0.0, (length * f / (2 * math.pi) - 1) / 31))
                f *= keep + (1 - keep) / factor
            out.append(f)
    return out


@pytest.mark.parametrize("size,axes,pairs", [(2, 1, [1]), (128, 1, [64]), (64, 3, [11, 11, 10]), (28, 2, [7, 7]),
                                             (4, 3, [1, 1, 0]), (256, 3, [43, 43, 42])])
@pytest.mark.parametrize("scaling", [None, "linear", "base", "parts"])
def test_steps(lib, size, axes, pairs, scaling):
    import sparse_convolution_gb300 as fvx

    more = dict(scaling=scaling, factor=8.0) if scaling else {}
    if scaling == "parts":
        more["length"] = 4096
    r = fvx.Rotary(size, axes=axes, base=5e5, **more)
    want = np.asarray(_frequencies(pairs, 5e5, scaling, 8.0, 4096)) / (2 * math.pi)
    # 64-bit powers, products and quotients: a few halves of 2^-52 each, and the step of the integers
    assert np.all(np.abs(r.turns.astype(np.float64) / 2.0 ** 64 - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -64)
    assert r.magnitude == pytest.approx(0.1 * math.log(8) + 1 if scaling == "parts" else 1.0, rel=2.0 ** -23)


@pytest.mark.parametrize("bad", [dict(size=3), dict(size=0), dict(size=258), dict(axes=4), dict(axes=0),
                                 dict(layout="both"), dict(scaling="other"), dict(scaling="parts"), dict(length=5),
                                 dict(base=1.0), dict(base=float("nan")), dict(scaling="linear", factor=0.5),
                                 dict(scaling="base", factor=float("inf")), dict(scaling="parts", length=0.0)])
def test_rotary_refuses(lib, bad):
    import sparse_convolution_gb300 as fvx

    with pytest.raises(fvx.FvxError) as e:
        fvx.Rotary(**{**dict(size=8), **bad})
    assert e.value.status == "FVX_ERR_INVALID_ARG"


def test_copies_own_their_steps(lib):
    """A copied or unpickled Rotary does not point into the original's memory."""
    import copy
    import gc
    import pickle

    import sparse_convolution_gb300 as fvx

    r = fvx.Rotary(64, axes=2, layout="interleaved", scaling="parts", factor=4.0, length=1000)
    want, copies = r.turns.copy(), [copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))]
    assert not r.turns.flags.writeable
    del r
    gc.collect()
    for c in copies:
        held = np.ctypeslib.as_array(ctypes.cast(c._struct.turns, ctypes.POINTER(ctypes.c_uint64)), (32,))
        assert np.array_equal(held, want) and c._struct.turns == c.turns.ctypes.data
        assert c._at == ctypes.addressof(c._struct) and (c.axes, c.layout, c.size) == (2, "interleaved", 64)
        assert c.magnitude == pytest.approx(0.1 * math.log(4) + 1, rel=2.0 ** -23)


def test_turns_refuses(lib):
    f = lib.fvx_rotary_turns
    turns, m = (ctypes.c_uint64 * 128)(), ctypes.c_float()
    three = lambda *p: (ctypes.c_int32 * 3)(*p)  # noqa: E731
    assert f(three(128, 0, 0), 1e4, 0, 1.0, 0.0, turns, ctypes.byref(m)) == OK
    for args in ((None, 1e4, 0, 1.0, 0.0, turns, ctypes.byref(m)), (three(4, 0, 0), 1e4, 0, 1.0, 0.0, None, ctypes.byref(m)),
                 (three(4, 0, 0), 1e4, 0, 1.0, 0.0, turns, None), (three(0, 0, 0), 1e4, 0, 1.0, 0.0, turns, ctypes.byref(m)),
                 (three(-1, 4, 0), 1e4, 0, 1.0, 0.0, turns, ctypes.byref(m)),
                 (three(100, 29, 0), 1e4, 0, 1.0, 0.0, turns, ctypes.byref(m)),
                 (three(4, 0, 0), 1e4, 4, 1.0, 0.0, turns, ctypes.byref(m)),
                 (three(4, 0, 0), 1e4, -1, 1.0, 0.0, turns, ctypes.byref(m))):
        assert f(*args) == INVALID, args
    assert b"fvx_rotary_turns" in lib.fvx_last_error()


# ---------------------------------------------------------------- heads
FIELDS = ("n", "heads", "in_", "in_token", "in_head", "out", "out_token", "out_head", "positions", "pos_token",
          "pos_axis", "weight", "x", "x_token", "x_head", "dweight")
GOOD = dict(n=5, heads=2, in_=P, in_token=128, in_head=64, out=P, out_token=128, out_head=64, positions=P, pos_token=1,
            pos_axis=0, weight=P, x=P, x_token=128, x_head=64, dweight=P)


def _rotary(pairs=(32, 0, 0), turns=True, magnitude=1.0):
    import sparse_convolution_gb300 as fvx

    s = fvx._RotaryStruct()
    s.pairs[0], s.pairs[1], s.pairs[2] = pairs
    s.magnitude = magnitude
    keep = (ctypes.c_uint64 * 256)()
    s.turns = ctypes.addressof(keep) if turns else None
    return s, keep


def _call(lib, entry, dt=1, d=64, count=1, rotary=None, last=1e-6, no_rotary=False, **change):
    t = {**GOOD, **change}
    packed = struct.pack("2qP2qP2qP2qPP2qP", *(t[f] for f in FIELDS)) * 2
    s, keep = rotary or _rotary()
    at = None if no_rotary else ctypes.addressof(s)
    f = getattr(lib, entry)
    return f(dt, d, packed, count, at, int(last) if entry == "fvx_rotate_heads" else last, None)


ENTRIES = ["fvx_rotate_heads", "fvx_norm_rotate_heads", "fvx_norm_rotate_heads_backward"]
BAD = [dict(dt=2), dict(d=0), dict(d=257), dict(count=0), dict(count=3), dict(n=-1), dict(heads=0), dict(in_=0),
       dict(out=0), dict(in_=P + 1), dict(out=P + 1), dict(in_token=-1), dict(in_head=-64), dict(out_token=-128),
       dict(positions=0), dict(positions=P + 2), dict(pos_token=-1), dict(weight=P + 2), dict(dweight=P + 1),
       dict(out_token=0), dict(out_head=0), dict(out_head=63), dict(out_token=127), dict(d=62)]


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("change", BAD)
def test_heads(lib, entry, change):
    assert _call(lib, entry, **change) == INVALID
    assert entry.encode() + b":" in lib.fvx_last_error()


@pytest.mark.parametrize("entry", ENTRIES)
def test_rotary_struct(lib, entry):
    for r in (_rotary(turns=False), _rotary((0, 0, 0)), _rotary((33, 0, 0)), _rotary((40, -8, 0)),
              _rotary(magnitude=float("nan")), _rotary(magnitude=float("inf"))):
        assert _call(lib, entry, rotary=r) == INVALID
    assert _call(lib, entry, rotary=_rotary((11, 11, 10)), pos_axis=-1) == INVALID
    assert _call(lib, entry, n=(1 << 30) // 2 + 1) == RANGE


def test_norm_and_backward(lib):
    for entry in ENTRIES[1:]:
        for eps in (-1.0, float("nan")):
            assert _call(lib, entry, last=eps) == INVALID
    assert _call(lib, ENTRIES[0], no_rotary=True) == INVALID
    for change in (dict(x=0), dict(x=P + 1), dict(x_token=-1), dict(x_head=-1)):
        assert _call(lib, ENTRIES[2], **change) == INVALID, change


def test_nothing_to_do(lib):
    """No tokens, no rows: no launch, no pointer needed."""
    n0 = lib.fvx_launch_count()
    for entry in ENTRIES:
        assert _call(lib, entry, n=0, in_=0, out=0, positions=0, x=0, dweight=0, count=2) == OK
    assert lib.fvx_dropout(0, None, 8, None, 0, 0, 8, 0.5, 1, 2, None, None, 8, None) == OK
    assert lib.fvx_launch_count() == n0


# ---------------------------------------------------------------- dropout
@pytest.mark.parametrize("change", [dict(dt=2), dict(x=None), dict(y=None), dict(x=P + 1), dict(y=P + 1), dict(r=P + 1),
                                    dict(n=-1), dict(c=0), dict(c=1 << 31, ldx=1 << 32, ldy=1 << 31, ldr=1 << 31),
                                    dict(p=-0.01), dict(p=1.01), dict(p=float("nan")), dict(ldx=31), dict(ldy=31),
                                    dict(ldr=31), dict(state=P + 4), dict(n=1 << 59, c=32)])
def test_dropout(lib, change):
    a = {**dict(dt=1, x=P, ldx=32, r=P, ldr=32, n=4, c=32, p=0.1, state=None, y=P, ldy=32), **change}
    st = lib.fvx_dropout(a["dt"], a["x"], a["ldx"], a["r"], a["ldr"], a["n"], a["c"], a["p"], 1, 2, a["state"], a["y"],
                         a["ldy"], None)
    assert st == INVALID
    assert b"fvx_dropout:" in lib.fvx_last_error()


def test_the_generator_of_the_tests():
    """The test suite's own Philox4x32-10 gives the vectors published with it."""
    ones = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((ones,) * 4, (ones,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        got = philox(np.asarray([counter], np.uint64).T, *key)
        assert tuple(int(w[0]) for w in got) == want
