"""The C entry points of layer norm, checkpoints and cross attention refuse
malformed arguments on the host, before any CUDA work (no GPU needed)."""
import ctypes

import numpy as np
import pytest

INVALID, RANGE, OK = 1, 2, 0
P = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from sparse_convolution_gb300 import build_lib

    build_lib.build()
    import sparse_convolution_gb300 as fvx

    return fvx.load()


def _norm(lib, dt=0, x=P, ldx=32, n=4, c=32, w=P, b=P, eps=1e-5, y=P, ldy=32, mean=P, rstd=P, group=0, codes=None,
          steps=None):
    return lib.fvx_layer_norm(dt, x, ldx, n, c, w, b, eps, y, ldy, mean, rstd, group, codes, steps, None)


@pytest.mark.parametrize("change", [dict(dt=2), dict(x=None), dict(x=P + 1), dict(ldx=31), dict(n=-1), dict(c=0),
                                    dict(c=65537, ldx=70000, ldy=70000), dict(w=P + 2), dict(eps=-1.0),
                                    dict(eps=float("nan")), dict(y=None), dict(ldy=8), dict(mean=None),
                                    dict(rstd=None), dict(group=16), dict(group=32), dict(group=32, codes=P)])
def test_layer_norm(lib, change):
    assert _norm(lib, **change) == INVALID
    assert b"fvx_layer_norm" in lib.fvx_last_error()


def test_nothing_to_do(lib):
    """No rows: no launch, no pointer needed."""
    n0 = lib.fvx_launch_count()
    assert _norm(lib, n=0, x=None, y=None, mean=None, rstd=None) == OK
    assert lib.fvx_checkpoint_pack(1, None, 8, 0, 8, 64, None, None, None) == OK
    assert _attend(lib, q=None, out=None, lse=None, qo=(0, 0)) == OK
    assert lib.fvx_launch_count() == n0


def _norm_backward(lib, dt=0, dy=P, lddy=32, x=P, ldx=32, group=0, codes=None, steps=None, n=4, c=32, w=P, mean=P,
                   rstd=P, dx=P, lddx=32, dw=P, db=P):
    return lib.fvx_layer_norm_backward(dt, dy, lddy, x, ldx, group, codes, steps, n, c, w, mean, rstd, dx, lddx, dw, db,
                                       None)


@pytest.mark.parametrize("change", [dict(dt=7), dict(dy=None), dict(x=None), dict(lddy=3), dict(ldx=3), dict(dx=None),
                                    dict(lddx=3), dict(mean=None), dict(rstd=P + 2), dict(dw=P + 1), dict(db=P + 1),
                                    dict(group=32, codes=P, steps=P), dict(group=32, x=None),
                                    dict(group=8, x=None, codes=P, steps=P), dict(n=-2), dict(c=0)])
def test_layer_norm_backward(lib, change):
    assert _norm_backward(lib, **change) == INVALID
    assert b"fvx_layer_norm_backward" in lib.fvx_last_error()


def test_checkpoint(lib):
    pack, restore = lib.fvx_checkpoint_pack, lib.fvx_checkpoint_restore
    for args in ((0, None, 32, 4, 32, 64, P, P), (0, P, 8, 4, 32, 64, P, P), (0, P, 32, 4, 32, 63, P, P),
                 (0, P, 32, 4, 32, 64, None, P), (0, P, 32, 4, 32, 64, P, None), (5, P, 32, 4, 32, 64, P, P),
                 (0, P + 2, 32, 4, 32, 64, P, P)):
        assert pack(*args, None) == INVALID, args
    for args in ((0, 64, None, P, 4, 32, None, None, None, None, P, 32), (0, 64, P, P, 4, 32, P, None, None, None, P, 32),
                 (0, 64, P, P, 4, 32, None, None, P, None, P, 32), (0, 64, P, P, 4, 32, None, None, None, None, None, 32),
                 (0, 64, P, P, 4, 32, None, None, None, None, P, 31), (0, 0, P, P, 4, 32, None, None, None, None, P, 32)):
        assert restore(*args, None) == INVALID, args
    assert b"fvx_checkpoint_restore" in lib.fvx_last_error()



def _attend(lib, dt=1, q=P, k=P, v=P, st=(128, 64), qo=(0, 5), ko=(0, 7), B=1, heads=2, kv_heads=2, d=64, mask=None,
            scale=1.0, out=P, lse=P):
    qo, ko = (np.asarray(o, np.int64) if o is not None else None for o in (qo, ko))
    at = lambda o: o.ctypes.data_as(ctypes.c_void_p) if o is not None else None  # noqa: E731
    return lib.fvx_cross_attention(dt, q, *st, k, *st, v, *st, at(qo), at(ko), B, heads, kv_heads, d, mask, scale, out,
                                   lse, None)


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=P + 1), INVALID),
    (dict(st=(-128, 64)), INVALID), (dict(st=(128, -64)), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID),
    (dict(qo=(1, 5)), INVALID), (dict(qo=(0, 6, 5), ko=(0, 1, 2), B=2), INVALID), (dict(B=0), INVALID),
    (dict(heads=3), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(d=0), INVALID),
    (dict(d=129), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(out=P + 8), INVALID), (dict(lse=P + 2), INVALID),
    (dict(qo=(0, 1 << 30)), RANGE), (dict(ko=(0, 1 << 40)), RANGE)])
def test_cross_attention(lib, change, status):
    assert _attend(lib, **change) == status
    assert b"fvx_cross_attention" in lib.fvx_last_error()


def test_cross_attention_backward(lib):
    qo, ko = np.asarray([0, 5], np.int64), np.asarray([0, 7], np.int64)
    at = lambda o: o.ctypes.data_as(ctypes.c_void_p)  # noqa: E731

    def call(dout=P, q=P, out=P, lse=P, dq=P, dk=P, dv=P, d=64):
        return lib.fvx_cross_attention_backward(1, dout, 128, 64, q, 128, 64, P, 128, 64, P, 128, 64, out, lse, at(qo),
                                                at(ko), 1, 2, 2, d, None, 1.0, dq, dk, dv, None)

    for change in (dict(dout=None), dict(q=None), dict(out=None), dict(lse=None), dict(dq=None), dict(dk=None),
                   dict(dv=None), dict(d=200), dict(dq=P + 4), dict(dk=P + 8), dict(dv=P + 2)):
        assert call(**change) == INVALID, change
    assert b"fvx_cross_attention_backward" in lib.fvx_last_error()
