"""Binding of the operators around a recurrent state (``include/gdnq_layer.h``):
short causal convolution, selective state space scan, gated norm, residual norm.

Argument marshalling only, as in the package itself.  Token tensors are 2-D
(one row per token; the row distance is the tensor's own), or 3-D with the
heads as the middle dimension; descriptors are the dataclasses below or their
marshalled form (``.c()``).  Device pointers given as integers stand for
contiguous rows.
"""
from __future__ import annotations

import ctypes
import dataclasses

from . import EINVAL, IO_BF16, IO_F32, GdnqError, _check, _stream, lib

CONV_SILU = 1
SSM_SOFTPLUS = 1
NORM_GATE_SIGMOID, NORM_GATE_FIRST, NORM_GROUP_WEIGHT, NORM_RES_F32 = 1, 2, 4, 8

_i32, _u32, _i64, _f32, _P = ctypes.c_int32, ctypes.c_uint32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class _ConvDesc(ctypes.Structure):
    _fields_ = [("C", _i32), ("width", _i32), ("io_dtype", _i32), ("flags", _u32)]


class _SsmDesc(ctypes.Structure):
    _fields_ = [("H", _i32), ("dk", _i32), ("dv", _i32), ("hk", _i32), ("io_dtype", _i32), ("flags", _u32),
                ("dt_min", _f32), ("dt_max", _f32)]


class _SsmIo(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "B", "C", "dt", "y", "A", "D", "dt_bias")]
    _fields_ += [(n, _i64) for n in ("ldx", "ldb", "ldc", "lddt", "ldy")]


class _NormDesc(ctypes.Structure):
    _fields_ = [("D", _i32), ("group", _i32), ("io_dtype", _i32), ("flags", _u32), ("eps", _f32), ("w_offset", _f32)]


@dataclasses.dataclass
class ConvDesc:
    """Mirror of gdnq_conv_desc."""
    C: int
    width: int = 4
    io_dtype: int = IO_BF16
    flags: int = CONV_SILU

    def c(self) -> _ConvDesc:
        return _ConvDesc(*dataclasses.astuple(self))


@dataclasses.dataclass
class SsmDesc:
    """Mirror of gdnq_ssm_desc."""
    H: int
    dk: int = 128
    dv: int = 64
    hk: int = 0
    io_dtype: int = IO_BF16
    flags: int = SSM_SOFTPLUS
    dt_min: float = 0.0
    dt_max: float = float("inf")

    def c(self) -> _SsmDesc:
        return _SsmDesc(*dataclasses.astuple(self))


@dataclasses.dataclass
class NormDesc:
    """Mirror of gdnq_norm_desc."""
    D: int
    group: int = 0
    io_dtype: int = IO_BF16
    flags: int = 0
    eps: float = 1e-6
    w_offset: float = 0.0

    def c(self) -> _NormDesc:
        return _NormDesc(*dataclasses.astuple(self))


def _load():
    D, S, N = ctypes.POINTER(_ConvDesc), ctypes.POINTER(_SsmDesc), ctypes.POINTER(_NormDesc)
    io = ctypes.POINTER(_SsmIo)
    sig = {
        "gdnq_conv_prefill": [D, _P, _i64, _P, _P, _P, _i32, _P, _P, _P, _i32, _i32, _P, _i64, _P],
        "gdnq_conv_step": [D, _P, _i64, _P, _P, _P, _i32, _P, _i32, _P, _i64, _P],
        "gdnq_ssm_workspace": [S, _i32, _i32, ctypes.POINTER(ctypes.c_size_t)],
        "gdnq_ssm_prefill": [S, io, _P, _i32, _P, _P, _P, _i32, _i32, _P, ctypes.c_size_t, _P],
        "gdnq_ssm_step": [S, io, _P, _i32, _P, _i32, _P],
        "gdnq_norm_gated": [N, _P, _i64, _P, _i64, _P, _P, _i64, _i32, _P],
        "gdnq_norm_residual": [N, _P, _i64, _P, _f32, _P, _i64, _P, _i64, _P, _P, _i64, _i32, _P],
    }
    for name, args in sig.items():
        if not hasattr(lib, name):
            raise ImportError(f"the built library does not export {name}: it predates its sources; rebuild it "
                              "with __graft_entry__.build()")
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int


_load()


def _desc(d):
    return d if isinstance(d, ctypes.Structure) else d.c()


def _bad(msg):
    raise GdnqError(EINVAL, msg)


_torch = None
_dtypes = {}
_device = _raw_stream = None   # torch's own queries, without their Python wrappers where it has them


def _begin(stream):
    """(current device, stream handle) of a call.  Loads torch on first use;
    device -2 as long as no GPU is in use (no tensor is on it then)."""
    global _torch, _device, _raw_stream
    if _device is None:
        if _torch is None:
            import torch
            _dtypes.update({IO_F32: torch.float32, IO_BF16: torch.bfloat16})
            _torch = torch
        if not _torch.cuda.is_initialized():
            return -2, _stream(stream)
        _raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
        _device = getattr(_torch._C, "_cuda_getDevice", _torch.cuda.current_device)
    cur = _device()
    if stream is None:
        return cur, (_raw_stream(cur) if _raw_stream else _stream(None))
    return cur, _stream(stream)


def _refuse(t, dtype, cur, name):
    where = t.get_device()
    if where < 0:
        _bad(f"{name} is on {t.device}, not on a GPU")
    if where != cur:
        _bad(f"{name} is on {t.device}, not on the current device {cur}")
    if dtype is not None and t.dtype is not dtype:
        _bad(f"{name} is {t.dtype}, not {dtype}")


def _rows(t, n, width, dtype, cur, name):
    """(pointer, row distance) of n rows of `width` values."""
    if t is None or type(t) is int:
        return t, 0
    shape, st = t.shape, t.stride()
    if len(shape) == 2 and shape[1] == width and shape[0] >= n and t.dtype is dtype and t.get_device() == cur \
            and st[1] == 1 and st[0] >= width:
        return t.data_ptr(), st[0]
    _refuse(t, dtype, cur, name)
    if len(shape) == 3:
        flat = shape[1] * shape[2] == width and st[2] == 1 and (st[1] == shape[2] or shape[1] == 1)
    else:
        flat = len(shape) == 2 and shape[1] == width and (st[1] == 1 or width == 1)
    if not flat:
        _bad(f"{name} must have rows of {width} consecutive values (got shape {tuple(shape)}, strides {st})")
    if shape[0] < n:
        _bad(f"{name} has {shape[0]} rows, {n} are needed")
    # one row has no distance; a zero distance would read as "contiguous"
    if shape[0] > 1 and st[0] < width:
        _bad(f"the rows of {name} overlap")
    return t.data_ptr(), (st[0] if shape[0] > 1 else width)


def _flat(t, n, dtype, cur, name):
    """Pointer of at least n contiguous values."""
    if t is None or type(t) is int:
        return t
    if t.dtype is dtype and t.get_device() == cur and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    _refuse(t, dtype, cur, name)
    if not t.is_contiguous():
        _bad(f"{name} must be contiguous")
    _bad(f"{name} has {t.numel()} values, {n} are needed")


def _types(d):
    """The io, fp32 and int32 types of a call (an unknown io_dtype is the library's to refuse)."""
    return _dtypes.get(d.io_dtype, _torch.float32), _torch.float32, _torch.int32


def gdnq_conv_prefill(desc, x, w, bias, state, n_slots, slots, cont, cu_seqlens, n_seqs, T, y, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    io, f32, i32 = _types(d)
    C, width = d.C, d.width
    xp, ldx = _rows(x, T, C, io, cur, "x")
    yp, ldy = _rows(y, T, C, io, cur, "y")
    rc = lib.gdnq_conv_prefill(
        d, xp, ldx, _flat(w, width * C, f32, cur, "w"), _flat(bias, C, f32, cur, "bias"),
        _flat(state, n_slots * (width - 1) * C, io, cur, "state"), n_slots, _flat(slots, n_seqs, i32, cur, "slots"),
        _flat(cont, n_seqs, i32, cur, "cont"), _flat(cu_seqlens, n_seqs + 1, i32, cur, "cu_seqlens"), n_seqs, T, yp,
        ldy, st)
    if rc:
        _check(rc)


def gdnq_conv_step(desc, x, w, bias, state, n_slots, slots, n, y, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    io, f32, i32 = _types(d)
    C, width = d.C, d.width
    xp, ldx = _rows(x, n, C, io, cur, "x")
    yp, ldy = _rows(y, n, C, io, cur, "y")
    rc = lib.gdnq_conv_step(
        d, xp, ldx, _flat(w, width * C, f32, cur, "w"), _flat(bias, C, f32, cur, "bias"),
        _flat(state, n_slots * (width - 1) * C, io, cur, "state"), n_slots, _flat(slots, n, i32, cur, "slots"), n, yp,
        ldy, st)
    if rc:
        _check(rc)


def gdnq_ssm_workspace(desc, n_seqs, T) -> int:
    """Bytes of workspace that gdnq_ssm_prefill needs."""
    out = ctypes.c_size_t()
    _check(lib.gdnq_ssm_workspace(_desc(desc), n_seqs, T, ctypes.byref(out)))
    return out.value


def _ssm_io(d, cur, n, x, B, C, dt, A, D, dt_bias, y):
    io, f32, _ = _types(d)
    H = d.H
    nb, nx = (d.hk or H) * d.dk, H * d.dv
    xp, ldx = _rows(x, n, nx, io, cur, "x")
    bp, ldb = _rows(B, n, nb, io, cur, "B")
    cp, ldc = _rows(C, n, nb, io, cur, "C")
    tp, lddt = _rows(dt, n, H, io, cur, "dt")
    yp, ldy = _rows(y, n, nx, io, cur, "y")
    return _SsmIo(xp, bp, cp, tp, yp, _flat(A, H, f32, cur, "A"), _flat(D, H, f32, cur, "D"),
                  _flat(dt_bias, H, f32, cur, "dt_bias"), ldx, ldb, ldc, lddt, ldy)


def gdnq_ssm_prefill(desc, x, B, C, dt, A, D, dt_bias, y, S, n_slots, slots, cont, cu_seqlens, n_seqs, T,
                     workspace=None, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    _, f32, i32 = _types(d)
    nb = 0
    if type(workspace) is int:
        nb = gdnq_ssm_workspace(d, n_seqs, T)
    elif workspace is not None:
        _refuse(workspace, None, cur, "workspace")
        if not workspace.is_contiguous():
            _bad("workspace must be contiguous")
        nb = workspace.numel() * workspace.element_size()
        workspace = workspace.data_ptr()
    rc = lib.gdnq_ssm_prefill(
        d, _ssm_io(d, cur, T, x, B, C, dt, A, D, dt_bias, y), _flat(S, n_slots * d.H * d.dk * d.dv, f32, cur, "S"),
        n_slots, _flat(slots, n_seqs, i32, cur, "slots"), _flat(cont, n_seqs, i32, cur, "cont"),
        _flat(cu_seqlens, n_seqs + 1, i32, cur, "cu_seqlens"), n_seqs, T, workspace, nb, st)
    if rc:
        _check(rc)


def gdnq_ssm_step(desc, x, B, C, dt, A, D, dt_bias, y, S, n_slots, slots, n, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    _, f32, i32 = _types(d)
    rc = lib.gdnq_ssm_step(
        d, _ssm_io(d, cur, n, x, B, C, dt, A, D, dt_bias, y), _flat(S, n_slots * d.H * d.dk * d.dv, f32, cur, "S"),
        n_slots, _flat(slots, n, i32, cur, "slots"), n, st)
    if rc:
        _check(rc)


def gdnq_norm_gated(desc, x, z, w, y, rows, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    io, f32, _ = _types(d)
    D = d.D
    xp, ldx = _rows(x, rows, D, io, cur, "x")
    zp, ldz = _rows(z, rows, D, io, cur, "z")
    yp, ldy = _rows(y, rows, D, io, cur, "y")
    nw = (d.group or D) if d.flags & NORM_GROUP_WEIGHT else D
    rc = lib.gdnq_norm_gated(d, xp, ldx, zp, ldz, _flat(w, nw, f32, cur, "w"), yp, ldy, rows, st)
    if rc:
        _check(rc)


def gdnq_norm_residual(desc, x, post_w, scale, res, res_out, w, y, rows, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    io, f32, _ = _types(d)
    rio = f32 if d.flags & NORM_RES_F32 else io
    D = d.D
    xp, ldx = _rows(x, rows, D, io, cur, "x")
    rp, ldr = _rows(res, rows, D, rio, cur, "res")
    op, ldro = (rp, ldr) if res_out is res else _rows(res_out, rows, D, rio, cur, "res_out")
    yp, ldy = _rows(y, rows, D, io, cur, "y")
    rc = lib.gdnq_norm_residual(d, xp, ldx, _flat(post_w, D, f32, cur, "post_w"), scale, rp, ldr, op, ldro,
                                _flat(w, D, f32, cur, "w"), yp, ldy, rows, st)
    if rc:
        _check(rc)
