"""fvx: sparse-voxel IndexGrid build, 3x3x3 kernel map and sparse convolution
on GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/fvx.h`` (argument
marshalling only; every step runs in the CUDA library ``libfvx.so``).  Torch
tensors supply device memory and the current CUDA stream.  There is no CPU
fallback: if the library is missing or no GPU is visible, calls raise.

Pages: "fVDB: A Deep-Learning Framework for Sparse, Large Scale, and High
Performance Spatial Intelligence" (reading notes: IndexGrid, GPU-accelerated
IndexGrid build, Sparse-convolution operators) and "DriveRT" (Shared neighbour
maps, Kernels selected per GPU).
"""
from __future__ import annotations

import array
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfvx.so")

_lib = None

FVX_F32, FVX_BF16, FVX_BF16_OUT_BF16 = 0, 1, 2
FVX_CONV_AUTO, FVX_CONV_GATHER, FVX_CONV_LEAF, FVX_CONV_DIRECT, FVX_CONV_UNION, FVX_CONV_HALO = 0, 1, 2, 3, 4, 5


class FvxError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{status}: {message}")
        self.status = status


class GridView(ctypes.Structure):
    _fields_ = [("batch_size", ctypes.c_int32)] + [
        (n, ctypes.c_int64) for n in ("n_rows", "n_upper", "n_lower", "n_leaf", "n_active")
    ] + [(n, ctypes.c_void_p) for n in (
        "ijk", "row_to_index", "voxel_batch_offsets", "leaf_origin", "leaf_batch", "leaf_records",
        "lower_origin", "lower_batch", "lower_mask", "lower_prefix", "lower_first",
        "upper_origin", "upper_batch", "upper_mask", "upper_prefix", "upper_first")]


def load():
    """Loads ``libfvx.so`` (must have been built by ``__graft_entry__.build()``
    or ``build_lib.build()``).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FvxError("FVX_NOT_BUILT", f"{LIB_PATH} is missing; build the CUDA library first")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I32, U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64
    F32 = ctypes.c_float
    PP = ctypes.POINTER(ctypes.c_void_p)
    sigs = {
        "fvx_set_allocator": ([P, P, P], I32),
        "fvx_build_grid": ([P, I64, P, I32, P, PP], I32),
        "fvx_grid_counts": ([P, P, P, P, P], I32),
        "fvx_grid_view": ([P, ctypes.POINTER(GridView)], I32),
        "fvx_grid_batch_offsets": ([P, P], I32),
        "fvx_lookup": ([P, P, P, I64, P, P], I32),
        "fvx_coarsen": ([P, I32, P, PP], I32),
        "fvx_kernel_map": ([P, P, I32, I32, P, PP], I32),
        "fvx_kernel_map_transposed": ([P, P, I32, I32, P, PP], I32),
        "fvx_refine": ([P, I32, P, PP], I32),
        "fvx_kmap_view": ([P, PP, PP, PP, PP, P, P], I32),
        "fvx_sparse_conv": ([P, P, P, I32, P, I64, P, I64, P, P], I32),
        "fvx_sparse_conv_noalloc": ([P, P, P, I32, P, I64, P, I64, P, P], I32),
        "fvx_noalloc_status": ([P], I32),
        "fvx_testing_bounded_wait": ([I32, U64, P], I32),
        "fvx_sparse_conv_dgrad": ([P, P, P, I32, P, I64, P, I64, P, P], I32),
        "fvx_sparse_conv_wgrad": ([P, P, P, I32, P, I64, P, I64, P, P], I32),
        "fvx_voxels_along_rays": ([P, P, P, P, I64, ctypes.c_float, ctypes.c_float, P, PP], I32),
        "fvx_hits_view": ([P, PP, PP, PP, P, P], I32),
        "fvx_hits_destroy": ([P], I32),
        "fvx_layer_norm": ([I32, P, I64, I64, I64, P, P, F32, P, I64, P, P, I32, P, P, P], I32),
        "fvx_layer_norm_backward": ([I32, P, I64, P, I64, I32, P, P, I64, I64, P, P, P, P, I64, P, P, P], I32),
        "fvx_checkpoint_pack": ([I32, P, I64, I64, I64, I32, P, P, P], I32),
        "fvx_checkpoint_restore": ([I32, I32, P, P, I64, I64, P, P, P, P, P, I64, P], I32),
        "fvx_cross_attention": ([I32] + 3 * [P, I64, I64] + [P, P, I32, I32, I32, I32, P, F32, P, P, P], I32),
        "fvx_cross_attention_backward": ([I32] + 4 * [P, I64, I64] + [P, P, P, P, I32, I32, I32, I32, P, F32, P, P, P,
                                                                     P], I32),
        "fvx_grid_destroy": ([P], I32),
        "fvx_kmap_destroy": ([P], I32),
        "fvx_status_string": ([I32], ctypes.c_char_p),
        "fvx_last_error": ([], ctypes.c_char_p),
        "fvx_device_status": ([P], I32),
        "fvx_launch_count": ([], U64),
        "fvx_profile_enable": ([ctypes.c_char_p], I32),
        "fvx_profile_read": ([P, P], I32),
        "fvx_profile_read_each": ([P, ctypes.c_int64, P], I32),
        "fvx_set_conv_algo": ([I32], I32),
        "fvx_last_conv_algo": ([], I32),
        "fvx_last_conv_kernel": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _check(st):
    if st != 0:
        lib = load()
        raise FvxError(lib.fvx_status_string(st).decode(), lib.fvx_last_error().decode())


def _stream(stream=None):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


class _DevArray:
    """Zero-copy handle on library-owned device memory for torch.as_tensor."""

    def __init__(self, ptr, shape, typestr, owner):
        self.__cuda_array_interface__ = dict(shape=tuple(int(s) for s in shape), typestr=typestr,
                                             data=(int(ptr or 0), False), version=3, strides=None)
        self._owner = owner


_TYPESTR = {"i4": "<i4", "i8": "<i8", "u4": "<u4", "u8": "<u8", "f4": "<f4"}


def _view(ptr, shape, code, owner):
    import torch

    if any(int(s) == 0 for s in shape) or not ptr:
        dt = {"i4": torch.int32, "i8": torch.int64, "u4": torch.uint32, "u8": torch.uint64,
              "f4": torch.float32}[code]
        return torch.zeros(tuple(int(s) for s in shape), dtype=dt, device="cuda")
    t = torch.as_tensor(_DevArray(ptr, shape, _TYPESTR[code], owner), device="cuda")
    return t.clone()


class Grid:
    """A batch of IndexGrids built on the GPU (library-owned topology)."""

    def __init__(self, handle, stream=None):
        self._h = handle
        lib = load()
        c = (ctypes.c_int64 * 4)()
        _check(lib.fvx_grid_counts(self._h, ctypes.byref(c, 0), ctypes.byref(c, 8), ctypes.byref(c, 16),
                                   ctypes.byref(c, 24)))
        self.n_upper, self.n_lower, self.n_leaf, self.n_active = (int(v) for v in c)
        v = GridView()
        _check(lib.fvx_grid_view(self._h, ctypes.byref(v)))
        self.batch_size = int(v.batch_size)
        self.n_rows = int(v.n_rows)
        self._v = v

    @classmethod
    def build(cls, coords, batch_offsets=None, stream=None) -> "Grid":
        """coords: int32 CUDA tensor [N, 3]; batch_offsets: CSR int64 [B+1]
        (host sequence / numpy / CPU tensor), default one batch."""
        import torch

        assert coords.is_cuda and coords.dtype == torch.int32 and coords.dim() == 2 and coords.shape[1] == 3
        coords = coords.contiguous()
        n = coords.shape[0]
        if batch_offsets is None:
            batch_offsets = [0, n]
        offs = np.ascontiguousarray(np.asarray(batch_offsets, dtype=np.int64))
        h = ctypes.c_void_p()
        _check(load().fvx_build_grid(_ptr(coords), n, offs.ctypes.data_as(ctypes.c_void_p), len(offs) - 1,
                                     _stream(stream), ctypes.byref(h)))
        return cls(h)

    def destroy(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.fvx_grid_destroy(self._h)
            self._h = None

    __del__ = destroy

    def counts(self):
        return dict(n_upper=self.n_upper, n_lower=self.n_lower, n_leaf=self.n_leaf, n_active=self.n_active)

    def batch_offsets(self):
        out = np.zeros(self.batch_size + 1, np.int64)
        _check(load().fvx_grid_batch_offsets(self._h, out.ctypes.data_as(ctypes.c_void_p)))
        return out

    def topology(self):
        """Copies of every topology array as CUDA tensors."""
        v = self._v
        U, L, NL, NU = self.n_active, self.n_leaf, self.n_lower, self.n_upper
        return dict(
            ijk=_view(v.ijk, (U, 3), "i4", self), row_to_index=_view(v.row_to_index, (self.n_rows,), "i4", self),
            voxel_batch_offsets=_view(v.voxel_batch_offsets, (self.batch_size + 1,), "i8", self),
            leaf_origin=_view(v.leaf_origin, (L, 3), "i4", self), leaf_batch=_view(v.leaf_batch, (L,), "i4", self),
            leaf_records=_view(v.leaf_records, (L, 10), "u8", self),
            lower_origin=_view(v.lower_origin, (NL, 3), "i4", self),
            lower_batch=_view(v.lower_batch, (NL,), "i4", self), lower_mask=_view(v.lower_mask, (NL, 64), "u8", self),
            lower_prefix=_view(v.lower_prefix, (NL, 64), "u4", self),
            lower_first=_view(v.lower_first, (NL,), "u4", self),
            upper_origin=_view(v.upper_origin, (NU, 3), "i4", self),
            upper_batch=_view(v.upper_batch, (NU,), "i4", self),
            upper_mask=_view(v.upper_mask, (NU, 512), "u8", self),
            upper_prefix=_view(v.upper_prefix, (NU, 512), "u4", self),
            upper_first=_view(v.upper_first, (NU,), "u4", self))

    def ijk(self):
        return _view(self._v.ijk, (self.n_active, 3), "i4", self)

    def lookup(self, coords, batch=None, stream=None):
        import torch

        coords = coords.contiguous()
        out = torch.empty(coords.shape[0], dtype=torch.int32, device=coords.device)
        b = batch.contiguous() if batch is not None else None
        _check(load().fvx_lookup(self._h, _ptr(coords), _ptr(b), coords.shape[0], _ptr(out), _stream(stream)))
        return out

    def coarsen(self, stride=2, stream=None) -> "Grid":
        h = ctypes.c_void_p()
        _check(load().fvx_coarsen(self._h, int(stride), _stream(stream), ctypes.byref(h)))
        return Grid(h)

    def refine(self, factor=2, stream=None) -> "Grid":
        """Every voxel's factor^3 children (the refined grid)."""
        h = ctypes.c_void_p()
        _check(load().fvx_refine(self._h, int(factor), _stream(stream), ctypes.byref(h)))
        return Grid(h)


class KernelMap:
    """Per-offset (in, out) pair lists of a 3x3x3 kernel (library-owned)."""

    def __init__(self, gin: Grid, gout: Grid, stride=1, ksize=3, stream=None, transposed=False):
        """transposed: the map of the transposed convolution (output voxel q
        paired with the input p where stride * ijk(p) + d == ijk(q))."""
        h = ctypes.c_void_p()
        f = load().fvx_kernel_map_transposed if transposed else load().fvx_kernel_map
        _check(f(gin._h, gout._h, int(ksize), int(stride), _stream(stream), ctypes.byref(h)))
        self._h = h
        self.gin, self.gout, self.stride, self.transposed = gin, gout, int(stride), bool(transposed)
        ii, oo, mm = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
        nout = ctypes.c_int64()
        _check(_lib.fvx_kmap_view(h, None, ctypes.byref(ii), ctypes.byref(oo), ctypes.byref(mm), None,
                                  ctypes.byref(nout)))
        self.n_out = int(nout.value)
        self._ptrs = (ii.value, oo.value, mm.value)
        self._totals = None

    def _read_totals(self):
        # the list offsets stay on the device until first asked for (that read
        # synchronises the map's stream)
        if self._totals is None:
            offs, npairs = ctypes.c_void_p(), ctypes.c_int64()
            _check(_lib.fvx_kmap_view(self._h, ctypes.byref(offs), None, None, None, ctypes.byref(npairs), None))
            self._totals = (np.ctypeslib.as_array((ctypes.c_int64 * 28).from_address(offs.value)).copy(),
                            int(npairs.value))
        return self._totals

    @property
    def offsets(self):
        """HOST int64 [28]: list s is pairs [offsets[s], offsets[s+1])."""
        return self._read_totals()[0]

    @property
    def n_pairs(self):
        return self._read_totals()[1]

    def destroy(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.fvx_kmap_destroy(self._h)
            self._h = None

    __del__ = destroy

    def pairs(self):
        ii, oo, mm = self._ptrs
        return (_view(ii, (self.n_pairs,), "i4", self), _view(oo, (self.n_pairs,), "i4", self),
                _view(mm, (self.n_out,), "u4", self))


class Hits:
    """Active voxels along rays (library-owned CSR result of
    fvx_voxels_along_rays)."""

    def __init__(self, grid: Grid, origins, dirs, batch=None, tmin=0.0, tmax=float("inf"), stream=None):
        import torch

        assert origins.dtype == torch.float32 and dirs.dtype == torch.float32 and origins.is_cuda and dirs.is_cuda
        origins = origins.contiguous()
        dirs = dirs.contiguous()
        n = origins.shape[0]
        assert tuple(origins.shape) == (n, 3) and tuple(dirs.shape) == (n, 3)
        if batch is not None:
            batch = batch.to(torch.int32).contiguous()
        h = ctypes.c_void_p()
        _check(load().fvx_voxels_along_rays(grid._h, _ptr(origins), _ptr(dirs), _ptr(batch), n,
                                            ctypes.c_float(tmin), ctypes.c_float(tmax), _stream(stream),
                                            ctypes.byref(h)))
        self._h = h
        off, vox, t = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
        nh, nr = ctypes.c_int64(), ctypes.c_int64()
        _check(_lib.fvx_hits_view(h, ctypes.byref(off), ctypes.byref(vox), ctypes.byref(t), ctypes.byref(nh),
                                  ctypes.byref(nr)))
        self.n_hits, self.n_rays = int(nh.value), int(nr.value)
        self._ptrs = (off.value, vox.value, t.value)

    def arrays(self):
        """(offsets int64 [n_rays + 1], voxel int32 [n_hits], t float32 [n_hits, 2]), device copies."""
        off, vox, t = self._ptrs
        return (_view(off, (self.n_rays + 1,), "i8", self), _view(vox, (self.n_hits,), "i4", self),
                _view(t, (self.n_hits, 2), "f4", self))

    def destroy(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.fvx_hits_destroy(self._h)
            self._h = None

    __del__ = destroy


def sparse_conv(gin: Grid, gout: Grid, kmap: KernelMap, feats, W, out=None, out_dtype=None, stream=None):
    """out[q] = sum over pairs (p, q) of list s of feats[p] @ W[s].

    feats [gin.n_active, cin] and W [27, cin, cout]: both float32 (exact fp32
    FFMA, float32 out) or both bfloat16 (tensor cores, fp32 accumulation;
    out_dtype float32 by default, or bfloat16 for a rounded bf16 output)."""
    import torch

    assert feats.dtype == W.dtype and feats.is_cuda and W.is_cuda
    if feats.dtype == torch.float32:
        dt, odt = FVX_F32, torch.float32
    else:
        assert feats.dtype == torch.bfloat16
        odt = out_dtype or (out.dtype if out is not None else torch.float32)
        dt = {torch.float32: FVX_BF16, torch.bfloat16: FVX_BF16_OUT_BF16}[odt]
    feats = feats.contiguous()
    W = W.contiguous()
    cin, cout = W.shape[1], W.shape[2]
    assert W.shape[0] == 27 and feats.shape[1] == cin
    if out is None:
        out = torch.empty((gout.n_active, cout), dtype=odt, device=feats.device)
    assert out.dtype == odt and out.is_contiguous() and tuple(out.shape) == (gout.n_active, cout)
    _check(load().fvx_sparse_conv(gin._h, gout._h, kmap._h, dt, _ptr(feats), cin, _ptr(W), cout, _ptr(out),
                                  _stream(stream)))
    return out


def sparse_conv_dgrad(gin: Grid, gout: Grid, kmap_t: KernelMap, dout, W, out=None, out_dtype=None, stream=None):
    """Input gradient of sparse_conv(gin, gout, ...): dx [gin.n_active, cin].

    kmap_t: KernelMap(gout, gin, stride, transposed=True).  dout [gout.n_active,
    cout] and W [27, cin, cout] both float32 or both bfloat16 (float32 dx by
    default, bfloat16 with out_dtype=torch.bfloat16)."""
    import torch

    assert dout.dtype == W.dtype and dout.is_cuda and W.is_cuda
    if dout.dtype == torch.float32:
        dt, odt = FVX_F32, torch.float32
    else:
        assert dout.dtype == torch.bfloat16
        odt = out_dtype or (out.dtype if out is not None else torch.float32)
        dt = {torch.float32: FVX_BF16, torch.bfloat16: FVX_BF16_OUT_BF16}[odt]
    dout = dout.contiguous()
    W = W.contiguous()
    cin, cout = W.shape[1], W.shape[2]
    assert W.shape[0] == 27 and dout.shape[1] == cout
    if out is None:
        out = torch.empty((gin.n_active, cin), dtype=odt, device=dout.device)
    assert out.dtype == odt and out.is_contiguous() and tuple(out.shape) == (gin.n_active, cin)
    _check(load().fvx_sparse_conv_dgrad(gin._h, gout._h, kmap_t._h, dt, _ptr(dout), cout, _ptr(W), cin, _ptr(out),
                                        _stream(stream)))
    return out


def sparse_conv_wgrad(gin: Grid, gout: Grid, kmap: KernelMap, feats, dout, out=None, stream=None):
    """Weight gradient of sparse_conv(gin, gout, kmap, feats, W): float32
    [27, cin, cout].  feats and dout both float32 or both bfloat16."""
    import torch

    assert feats.dtype == dout.dtype and feats.is_cuda and dout.is_cuda
    dt = FVX_F32 if feats.dtype == torch.float32 else FVX_BF16
    assert dt == FVX_F32 or feats.dtype == torch.bfloat16
    feats = feats.contiguous()
    dout = dout.contiguous()
    cin, cout = feats.shape[1], dout.shape[1]
    if out is None:
        out = torch.empty((27, cin, cout), dtype=torch.float32, device=feats.device)
    assert out.dtype == torch.float32 and out.is_contiguous() and tuple(out.shape) == (27, cin, cout)
    _check(load().fvx_sparse_conv_wgrad(gin._h, gout._h, kmap._h, dt, _ptr(feats), cin, _ptr(dout), cout, _ptr(out),
                                        _stream(stream)))
    return out


# ---------------------------------------------------------------- layer norm, checkpoints, cross attention
def _refuse(message):
    raise FvxError("FVX_ERR_INVALID_ARG", message)


def _dtype_code(t, who):
    import torch

    if t.dtype == torch.bfloat16:
        return FVX_BF16
    if t.dtype != torch.float32:
        _refuse(f"{who}: tensors must be float32 or bfloat16, got {t.dtype}")
    return FVX_F32


def _on_device(who, *tensors):
    """Every tensor on the current CUDA device (the library launches there);
    returns the current stream's handle."""
    import torch

    dev = torch._C._cuda_getDevice() if tensors[0].is_cuda else torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _refuse(f"{who}: every tensor must be on the current CUDA device {dev}, got {t.device}")
    return torch._C._cuda_getCurrentRawStream(dev)


def _empty_rows(t):
    """Room for a result of t's shape and type, dense."""
    import torch

    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _on_stream(stream, call, *args, **kw):
    """call(*args, **kw) with `stream` current, so that what it allocates
    belongs to the stream its kernels run on."""
    import torch

    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _rows(t, who, name):
    """t as rows of dense channels: (tensor, pitch); a copy only where the channels are strided."""
    if t.dim() != 2:
        _refuse(f"{who}: {name} must be [rows, channels], got {tuple(t.shape)}")
    n, c = t.shape
    if c < 1:
        _refuse(f"{who}: {name} has no channels")
    if (c > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < c):
        t = t.contiguous()
    return t, (t.stride(0) if n > 1 else c)


def _channel_vector(t, c, who, name):
    import torch

    if t is None:
        return None
    if t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != c:
        _refuse(f"{who}: {name} must be float32 [{c}], got {t.dtype} {tuple(t.shape)}")
    return t if t.stride(0) == 1 or c == 1 else t.contiguous()


def _row_vector(t, n, who, name):
    import torch

    if t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != n:
        _refuse(f"{who}: {name} must be float32 [{n}], got {t.dtype} {tuple(t.shape)}")
    return t if t.is_contiguous() else t.contiguous()


def _at(t):
    return t.data_ptr() if t is not None else None


class Checkpoint8:
    """Activations [rows, channels] held in 8 bits: ``codes`` int8 and one fp32
    ``steps`` value per group of 32, 64 or 128 channels of a row; the value held
    is code * step, within half a step of the activation.

    Made by ``Checkpoint8.pack`` or by ``layer_norm(checkpoint_group=...)`` and
    read by ``restore``, by ``layer_norm`` (the norm's output computed again) and
    by ``layer_norm_backward``."""

    def __init__(self, codes, steps, group, dtype):
        self.codes, self.steps, self.group, self.dtype = codes, steps, group, dtype

    @staticmethod
    def _empty(x, group, who):
        import torch

        if group not in (32, 64, 128):
            _refuse(f"{who}: the checkpoint's group must be 32, 64 or 128, got {group}")
        n, c = x.shape
        return Checkpoint8(torch.empty((n, c), dtype=torch.int8, device=x.device),
                           torch.empty((n, -(-c // group)), dtype=torch.float32, device=x.device), group, x.dtype)

    @classmethod
    def pack(cls, x, group=64, stream=None) -> "Checkpoint8":
        """x: float32 or bfloat16 [rows, channels]."""
        if stream is not None:
            return _on_stream(stream, cls.pack, x, group)
        who = "Checkpoint8.pack"
        dt = _dtype_code(x, who)
        s = _on_device(who, x)
        x, ld = _rows(x, who, "x")
        ck = cls._empty(x, group, who)
        n, c = ck.codes.shape
        _check(load().fvx_checkpoint_pack(dt, x.data_ptr(), ld, n, c, group, ck.codes.data_ptr(), ck.steps.data_ptr(), s))
        return ck

    def _checked(self, who):
        """(codes, steps) after a look at whether they belong together: the
        attributes can be set by hand, and the kernels go by the codes' shape."""
        import torch

        codes, steps, group = self.codes, self.steps, self.group
        if group not in (32, 64, 128):
            _refuse(f"{who}: the checkpoint's group must be 32, 64 or 128, got {group}")
        if codes.dtype != torch.int8 or codes.dim() != 2 or not codes.is_contiguous():
            _refuse(f"{who}: the checkpoint's codes must be int8 [rows, channels], contiguous, "
                    f"got {codes.dtype} {tuple(codes.shape)}")
        want = (codes.shape[0], -(-codes.shape[1] // group))
        if steps.dtype != torch.float32 or tuple(steps.shape) != want or not steps.is_contiguous():
            _refuse(f"{who}: the checkpoint's steps must be float32 {list(want)}, contiguous, "
                    f"got {steps.dtype} {tuple(steps.shape)}")
        return codes, steps

    @property
    def shape(self):
        return self.codes.shape

    @property
    def nbytes(self):
        return self.codes.numel() + 4 * self.steps.numel()

    def _restore(self, who, parts, mean, rstd, weight, bias, dtype, out):
        import torch

        codes, steps = parts
        n, c = codes.shape
        if out is None:
            out = torch.empty((n, c), dtype=dtype or self.dtype, device=codes.device)
            ld = c
        else:
            if tuple(out.shape) != (n, c) or (c > 1 and out.stride(1) != 1) or (n > 1 and out.stride(0) < c):
                _refuse(f"{who}: out must be [{n}, {c}] with dense channels, got {tuple(out.shape)}")
            ld = out.stride(0) if n > 1 else c
        dt = _dtype_code(out, who)
        s = _on_device(who, codes, steps, mean, rstd, weight, bias, out)
        _check(load().fvx_checkpoint_restore(dt, self.group, codes.data_ptr(), steps.data_ptr(), n, c, _at(mean),
                                             _at(rstd), _at(weight), _at(bias), out.data_ptr(), ld, s))
        return out

    def restore(self, dtype=None, out=None, stream=None):
        """The values held, in the activations' type or ``dtype``."""
        if stream is not None:
            return _on_stream(stream, self.restore, dtype, out)
        who = "Checkpoint8.restore"
        return self._restore(who, self._checked(who), None, None, None, None, dtype, out)

    def layer_norm(self, mean, rstd, weight=None, bias=None, dtype=None, out=None, stream=None):
        """Layer norm of the values held, with the forward pass's statistics:
        the input of what followed the norm, for its backward pass."""
        if stream is not None:
            return _on_stream(stream, self.layer_norm, mean, rstd, weight, bias, dtype, out)
        who = "Checkpoint8.layer_norm"
        parts = self._checked(who)
        n, c = parts[0].shape
        mean, rstd = _row_vector(mean, n, who, "mean"), _row_vector(rstd, n, who, "rstd")
        weight, bias = _channel_vector(weight, c, who, "weight"), _channel_vector(bias, c, who, "bias")
        return self._restore(who, parts, mean, rstd, weight, bias, dtype, out)


def layer_norm(x, weight=None, bias=None, eps=1e-5, checkpoint_group=None, stream=None):
    """Layer norm of each row of x [rows, channels] (float32 or bfloat16);
    weight and bias float32 [channels] or None.  Returns (y, mean, rstd), the
    statistics float32 [rows]; with checkpoint_group (32, 64 or 128) also x's
    Checkpoint8, written by the same pass."""
    import torch

    if stream is not None:
        return _on_stream(stream, layer_norm, x, weight, bias, eps, checkpoint_group)
    who = "layer_norm"
    dt = _dtype_code(x, who)
    s = _on_device(who, x, weight, bias)
    x, ld = _rows(x, who, "x")
    n, c = x.shape
    weight, bias = _channel_vector(weight, c, who, "weight"), _channel_vector(bias, c, who, "bias")
    dev = x.device
    y = _empty_rows(x)
    mean = torch.empty((n,), dtype=torch.float32, device=dev)
    rstd = torch.empty((n,), dtype=torch.float32, device=dev)
    if not checkpoint_group:
        _check(load().fvx_layer_norm(dt, x.data_ptr(), ld, n, c, _at(weight), _at(bias), eps, y.data_ptr(), c,
                                     mean.data_ptr(), rstd.data_ptr(), 0, None, None, s))
        return y, mean, rstd
    ck = Checkpoint8._empty(x, checkpoint_group, who)
    _check(load().fvx_layer_norm(dt, x.data_ptr(), ld, n, c, _at(weight), _at(bias), eps, y.data_ptr(), c,
                                 mean.data_ptr(), rstd.data_ptr(), checkpoint_group, ck.codes.data_ptr(),
                                 ck.steps.data_ptr(), s))
    return y, mean, rstd, ck


def layer_norm_backward(dy, x, mean, rstd, weight=None, stream=None):
    """Gradients of layer_norm: (dx, dweight, dbias), dx in dy's type, the
    others float32 [channels].  x: the tensor given to layer_norm, or its
    Checkpoint8 (then x is read from its 8-bit codes)."""
    import torch

    if stream is not None:
        return _on_stream(stream, layer_norm_backward, dy, x, mean, rstd, weight)
    who = "layer_norm_backward"
    dt = _dtype_code(dy, who)
    ck = x if isinstance(x, Checkpoint8) else None
    if x.shape != dy.shape:
        _refuse(f"{who}: x is {tuple(x.shape)}, dy {tuple(dy.shape)}")
    if x.dtype != dy.dtype:
        _refuse(f"{who}: x is {x.dtype}, dy {dy.dtype}")
    dy, lddy = _rows(dy, who, "dy")
    n, c = dy.shape
    if ck:
        codes, steps = ck._checked(who)
        s = _on_device(who, dy, mean, rstd, weight, codes, steps)
        source = (None, c, ck.group, codes.data_ptr(), steps.data_ptr())
    else:
        s = _on_device(who, dy, mean, rstd, weight, x)
        x, ldx = _rows(x, who, "x")
        source = (x.data_ptr(), ldx, 0, None, None)
    mean, rstd = _row_vector(mean, n, who, "mean"), _row_vector(rstd, n, who, "rstd")
    weight = _channel_vector(weight, c, who, "weight")
    dev = dy.device
    dx = _empty_rows(dy)
    dw = torch.empty((c,), dtype=torch.float32, device=dev)
    db = torch.empty((c,), dtype=torch.float32, device=dev)
    _check(load().fvx_layer_norm_backward(dt, dy.data_ptr(), lddy, *source, n, c, _at(weight), mean.data_ptr(),
                                          rstd.data_ptr(), dx.data_ptr(), c, dw.data_ptr(), db.data_ptr(), s))
    return dx, dw, db


def _heads(t, who, name):
    """t [tokens, heads, d] with a dense last dimension: a copy where it is
    not, and where a bf16 tensor's base or a stride is no multiple of 16 bytes
    (the tensor cores' copies need that)."""
    if t.dim() != 3:
        _refuse(f"{who}: {name} must be [tokens, heads, size], got {tuple(t.shape)}")
    if t.is_contiguous():
        return t if t.dtype.itemsize == 4 or not t.data_ptr() & 15 else t.clone()
    st = t.stride()
    if (t.shape[2] > 1 and st[2] != 1) or (t.dtype.itemsize == 2 and
                                           ((st[0] | st[1] | (t.data_ptr() >> 1)) & 7 or not st[0] or not st[1])):
        t = t.contiguous()
    return t


def _host_offsets(o):
    return array.array("q", o)  # of ints, or of a tensor's or an array's elements


def _attention_args(who, q, k, v, q_offsets, kv_offsets, key_mask):
    import torch

    q, k, v = _heads(q, who, "q"), _heads(k, who, "k"), _heads(v, who, "v")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        _refuse(f"{who}: q, k and v must have one type, got {q.dtype}, {k.dtype}, {v.dtype}")
    nq, heads, d = q.shape
    nk, kv_heads, dk = k.shape
    if v.shape != k.shape or dk != d:
        _refuse(f"{who}: q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not belong together")
    B = len(q_offsets) - 1
    if B < 1 or len(kv_offsets) != B + 1:
        _refuse(f"{who}: q_offsets and kv_offsets must both have B + 1 values, B at least 1")
    if q_offsets[B] != nq or kv_offsets[B] != nk:
        _refuse(f"{who}: the offsets end at {int(q_offsets[B])} and {int(kv_offsets[B])}, the tensors at {nq} and {nk}")
    if key_mask is not None:
        if key_mask.dtype not in (torch.bool, torch.uint8) or tuple(key_mask.shape) != (nk,):
            _refuse(f"{who}: key_mask must be bool [{nk}], got {key_mask.dtype} {tuple(key_mask.shape)}")
        key_mask = key_mask.contiguous()
    return q, k, v, key_mask, _host_offsets(q_offsets), _host_offsets(kv_offsets), B


def cross_attention(q, k, v, q_offsets, kv_offsets, key_mask=None, scale=None, stream=None):
    """Attention from the query rows of each batch element to that element's
    keys.  q [nq, heads, size], k and v [nk, kv_heads, size], all float32 or
    all bfloat16, heads a multiple of kv_heads, size at most 128; q_offsets and
    kv_offsets: CSR [B + 1] over tokens (host sequences; Grid.batch_offsets()
    gives a grid's); key_mask: bool [nk], True = kept; scale: default
    1 / sqrt(size).  Returns (out [nq, heads, size], lse float32 [nq, heads]);
    a row without kept keys gets zeros and -inf."""
    import torch

    if stream is not None:
        return _on_stream(stream, cross_attention, q, k, v, q_offsets, kv_offsets, key_mask, scale)
    who = "cross_attention"
    dt = _dtype_code(q, who)
    s = _on_device(who, q, k, v, key_mask)
    q, k, v, key_mask, qo, ko, B = _attention_args(who, q, k, v, q_offsets, kv_offsets, key_mask)
    nq, heads, d = q.shape
    out = _empty_rows(q)
    lse = torch.empty((nq, heads), dtype=torch.float32, device=q.device)
    _check(load().fvx_cross_attention(dt, *_strided(q), *_strided(k), *_strided(v), qo.buffer_info()[0],
                                      ko.buffer_info()[0], B, heads, k.shape[1], d, _at(key_mask),
                                      d ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(), s))
    return out, lse


def cross_attention_backward(dout, q, k, v, out, lse, q_offsets, kv_offsets, key_mask=None, scale=None, stream=None):
    """Gradients (dq, dk, dv) of cross_attention, in the tensors' type, from
    dout and what cross_attention returned; a key head's gradients sum over the
    query heads that read it."""
    import torch

    if stream is not None:
        return _on_stream(stream, cross_attention_backward, dout, q, k, v, out, lse, q_offsets, kv_offsets, key_mask,
                          scale)
    who = "cross_attention_backward"
    dt = _dtype_code(q, who)
    s = _on_device(who, dout, q, k, v, out, lse, key_mask)
    q, k, v, key_mask, qo, ko, B = _attention_args(who, q, k, v, q_offsets, kv_offsets, key_mask)
    nq, heads, d = q.shape
    for name, t in (("dout", dout), ("out", out)):
        if t.dtype != q.dtype or t.shape != q.shape:
            _refuse(f"{who}: {name} must be {q.dtype} {tuple(q.shape)}, got {t.dtype} {tuple(t.shape)}")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (nq, heads):
        _refuse(f"{who}: lse must be float32 [{nq}, {heads}], got {lse.dtype} {tuple(lse.shape)}")
    dout, out, lse = _heads(dout, who, "dout"), out.contiguous(), lse.contiguous()
    if out.data_ptr() & 15:  # a part of something wider that the caller kept
        out = out.clone()
    dq, dk, dv = _empty_rows(q), _empty_rows(k), _empty_rows(k)
    _check(load().fvx_cross_attention_backward(
        dt, *_strided(dout), *_strided(q), *_strided(k), *_strided(v), out.data_ptr(), lse.data_ptr(),
        qo.buffer_info()[0], ko.buffer_info()[0], B, heads, k.shape[1], d, _at(key_mask),
        d ** -0.5 if scale is None else scale, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), s))
    return dq, dk, dv


def _strided(t):
    st = t.stride()
    return t.data_ptr(), st[0], st[1]


def device_status(stream=None):
    _check(load().fvx_device_status(_stream(stream)))


def noalloc_status(stream=None):
    """Status of the last fvx_sparse_conv_noalloc call (raises FvxError on a
    recorded timeout or check failure)."""
    _check(load().fvx_noalloc_status(_stream(stream)))


def set_conv_algo(algo: int) -> None:
    """FVX_CONV_AUTO (default), FVX_CONV_GATHER, FVX_CONV_DIRECT,
    FVX_CONV_UNION, FVX_CONV_HALO or FVX_CONV_LEAF: which bf16 convolution
    kernel sparse_conv runs (process-wide)."""
    _check(load().fvx_set_conv_algo(int(algo)))


def last_conv_algo() -> int:
    """FVX_CONV_GATHER, FVX_CONV_LEAF or FVX_CONV_HALO: what the last bf16
    convolution on this thread ran (FVX_CONV_AUTO before any)."""
    return int(load().fvx_last_conv_algo())


def last_conv_kernel() -> str:
    """Name of the kernel the last convolution on this thread launched."""
    return load().fvx_last_conv_kernel().decode()


def launch_count() -> int:
    return int(load().fvx_launch_count())


def profile_enable(kernel_name):
    _check(load().fvx_profile_enable(kernel_name.encode() if kernel_name else None))


def profile_read():
    ms, n = ctypes.c_double(), ctypes.c_int64()
    _check(load().fvx_profile_read(ctypes.byref(ms), ctypes.byref(n)))
    return float(ms.value), int(n.value)


def profile_read_each(cap=4096):
    """Durations (ms) of the timed launches, in launch order."""
    buf = (ctypes.c_double * cap)()
    n = ctypes.c_int64()
    _check(load().fvx_profile_read_each(buf, cap, ctypes.byref(n)))
    return [float(buf[i]) for i in range(min(cap, n.value))]
