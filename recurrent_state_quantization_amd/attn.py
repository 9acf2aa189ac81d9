"""Binding of the operators of a softmax attention layer around its paged cache
(``include/gdnq_attn.h``): rotary positions, storing new tokens, the attention
of one new token, eviction by accumulated weight.

Argument marshalling only, as in ``layer.py``, whose conventions hold.  The
cache is a :class:`Kv` of the caller's tensors; a program that repeats calls
marshals it once (``kv.c(desc)``) and keeps the tensors.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Any

from . import IO_BF16, _check, lib
from . import layer as _layer
from .layer import _bad, _begin, _desc, _flat, _refuse, _rows

ROPE_INTERLEAVED, ROPE_INVERSE = 1, 2
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_RAMP_TURNS, ROPE_RAMP_INDEX = 0, 1, 2, 3, 4

_i32, _u32, _i64, _f32, _f64, _P = (ctypes.c_int32, ctypes.c_uint32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                                    ctypes.c_void_p)


class _RopeDesc(ctypes.Structure):
    _fields_ = [("d", _i32), ("rot", _i32), ("io_dtype", _i32), ("flags", _u32), ("amp", _f32)]


class _RopeFreqs(ctypes.Structure):
    _fields_ = [("kind", _i32), ("base", _f64), ("factor", _f64), ("orig_len", _f64), ("lo", _f64), ("hi", _f64),
                ("divisors", ctypes.POINTER(_f64))]


class _AttnDesc(ctypes.Structure):
    _fields_ = [("H", _i32), ("hk", _i32), ("d", _i32), ("io_dtype", _i32), ("page", _i32), ("window", _i32),
                ("scale", _f32), ("acc_decay", _f32)]


class _Kv(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k", "v", "acc", "pos", "table", "lens")]
    _fields_ += [(n, _i32) for n in ("n_pages", "n_slots", "max_pages")]
    _fields_ += [(n, _i64) for n in ("ldp", "ldh", "ldr")]


@dataclasses.dataclass
class RopeDesc:
    """Mirror of gdnq_rope_desc."""
    d: int
    rot: int = 0
    io_dtype: int = IO_BF16
    flags: int = 0
    amp: float = 1.0

    def c(self) -> _RopeDesc:
        return _RopeDesc(*dataclasses.astuple(self))


@dataclasses.dataclass
class RopeFreqs:
    """Mirror of gdnq_rope_freqs; divisors is a sequence of rot/2 numbers, or None."""
    kind: int = ROPE_PLAIN
    base: float = 10000.0
    factor: float = 1.0
    orig_len: float = 0.0
    lo: float = 1.0
    hi: float = 32.0
    divisors: Any = None


@dataclasses.dataclass
class AttnDesc:
    """Mirror of gdnq_attn_desc."""
    H: int
    hk: int = 0
    d: int = 128
    io_dtype: int = IO_BF16
    page: int = 64
    window: int = 0
    scale: float = 0.0
    acc_decay: float = 1.0

    def c(self) -> _AttnDesc:
        return _AttnDesc(*dataclasses.astuple(self))


@dataclasses.dataclass
class Kv:
    """The cache: k and v [n_pages, hk, page, d] (any order of pages, heads and
    rows in memory, the same for both), table [n_slots, max_pages] and lens
    [n_slots] int32, acc fp32 and pos int32 [n_pages, hk, page] or None."""
    k: Any
    v: Any
    table: Any
    lens: Any
    acc: Any = None
    pos: Any = None

    def c(self, desc) -> _Kv:
        d = _desc(desc)
        cur, _ = _begin(0)
        io, f32, i32 = _layer._types(d)
        hk = d.hk or d.H
        for name in ("k", "v"):
            t = getattr(self, name)
            _refuse(t, io, cur, name)
            if t.dim() != 4 or tuple(t.shape[1:]) != (hk, d.page, d.d) or t.stride(3) != 1:
                _bad(f"{name} must be [n_pages, {hk}, {d.page}, {d.d}] with consecutive values in a row (got shape "
                     f"{tuple(t.shape)}, strides {t.stride()})")
        if self.v.shape != self.k.shape or any(
                a != b for a, b, m in zip(self.v.stride(), self.k.stride(), self.k.shape) if m > 1):
            _bad("v must have the shape and strides of k")
        if self.table.dim() != 2:
            _bad("table must be [n_slots, max_pages]")
        n, (slots, width) = self.k.shape[0], self.table.shape
        # a dimension of one has no distance: any that holds what is inside it
        st = self.k.stride()
        ldr = st[2] if d.page > 1 else d.d
        ldh = st[1] if hk > 1 else max(ldr * d.page, d.d)
        ldp = st[0] if n > 1 else max(ldh * hk, ldr * d.page)
        if min(ldr, ldh, ldp) < d.d:   # three of zero would read as the default layout
            _bad(f"the rows of k overlap (strides {st})")
        kv = _Kv(self.k.data_ptr(), self.v.data_ptr(), _flat(self.acc, n * hk * d.page, f32, cur, "acc"),
                 _flat(self.pos, n * hk * d.page, i32, cur, "pos"), _flat(self.table, slots * width, i32, cur, "table"),
                 _flat(self.lens, slots, i32, cur, "lens"),
                 n, slots, width, ldp, ldh, ldr)
        # what the pointers stand for, kept as long as they are, and checked by every call
        kv.tensors, kv.of, kv.device = self, (hk, d.d, d.io_dtype, d.page), cur
        return kv


def _load():
    R, A, K = ctypes.POINTER(_RopeDesc), ctypes.POINTER(_AttnDesc), ctypes.POINTER(_Kv)
    size = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "gdnq_rope_table": [R, ctypes.POINTER(_RopeFreqs), _P],
        "gdnq_rope": [R, _P, _P, _i64, _i32, _P, _P, _i64, _i32, _P],
        "gdnq_kv_append": [A, R, _P, K, _P, _i64, _P, _i64, _P, _i64, _P, _i64, _P, _P, _P, _i32, _i32, _P],
        "gdnq_attn_workspace": [A, K, _i32, size],
        "gdnq_attn_step": [A, K, _P, _i64, _P, _i64, _P, _i32, _P, ctypes.c_size_t, _P],
        "gdnq_kv_evict_workspace": [A, K, _i32, _i32, size],
        "gdnq_kv_evict": [A, K, _i32, _i32, _i32, _P, _i32, _P, ctypes.c_size_t, _P],
    }
    for name, args in sig.items():
        if not hasattr(lib, name):
            raise ImportError(f"the built library does not export {name}: it predates its sources; rebuild it "
                              "with __graft_entry__.build()")
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int


_load()


def _kv(kv, d, cur=None):
    """The marshalled cache, which must be of this descriptor's sizes (and on the current device)."""
    if not isinstance(kv, _Kv):
        return kv.c(d)
    if hasattr(kv, "of"):   # one of plain pointers says nothing of itself
        if kv.of != (d.hk or d.H, d.d, d.io_dtype, d.page):
            _bad(f"kv is a cache of hk, d, io_dtype and page {kv.of}, not of desc's")
        if cur is not None and kv.device != cur:
            _bad(f"kv is on device {kv.device}, not on the current device {cur}")
    return kv


def _table(table, d, cur):
    """Device pointer of the rot/2 frequencies (int64 or uint64 values)."""
    if table is None or type(table) is int:
        return table
    if str(table.dtype) not in ("torch.int64", "torch.uint64"):
        _bad(f"table is {table.dtype}, not torch.int64 or torch.uint64")
    return _flat(table, (d.rot or d.d) // 2, table.dtype, cur, "table")


def _space(ws, cur, size):
    """(pointer, bytes) of a workspace; `size` gives the bytes behind a plain pointer."""
    if ws is None:
        return None, 0
    if type(ws) is int:
        return ws, size()
    if ws.get_device() != cur:
        _refuse(ws, None, cur, "workspace")
    if not ws.is_contiguous():
        _bad("workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def gdnq_rope_table(desc, freqs: RopeFreqs):
    """The frequencies of the pairs, a torch.int64 tensor [rot/2] on the host
    (the bits of the library's uint64): copy it to the device once."""
    import torch

    d = _desc(desc)
    div = None
    if freqs.divisors is not None:
        div = (_f64 * len(freqs.divisors))(*freqs.divisors)
        if len(div) < (d.rot or d.d) // 2:
            _bad(f"divisors has {len(div)} values, {(d.rot or d.d) // 2} are needed")
    f = _RopeFreqs(freqs.kind, freqs.base, freqs.factor, freqs.orig_len, freqs.lo, freqs.hi, div)
    out = torch.zeros(max(1, (d.rot or d.d) // 2), dtype=torch.int64)
    _check(lib.gdnq_rope_table(d, f, out.data_ptr()))
    return out


def gdnq_rope(desc, table, x, pos, y, rows, H, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    io, _, i32 = _layer._types(d)
    xp, ldx = _rows(x, rows, H * d.d, io, cur, "x")
    yp, ldy = (xp, ldx) if y is x else _rows(y, rows, H * d.d, io, cur, "y")
    rc = lib.gdnq_rope(d, _table(table, d, cur), xp, ldx, H, _flat(pos, rows, i32, cur, "pos"), yp, ldy, rows, st)
    if rc:
        _check(rc)


def gdnq_kv_append(desc, rope, table, kv, q, q_out, k, v, pos, slots, cu_seqlens, n, T, stream=None):
    d = _desc(desc)
    r = None if rope is None else _desc(rope)
    cur, st = _begin(stream)
    io, _, i32 = _layer._types(d)
    H, hk, D = d.H, d.hk or d.H, d.d
    qp, ldq = _rows(q, T, H * D, io, cur, "q")
    op, ldqo = (qp, ldq) if q_out is q else _rows(q_out, T, H * D, io, cur, "q_out")
    kp, ldk = _rows(k, T, hk * D, io, cur, "k")
    vp, ldv = _rows(v, T, hk * D, io, cur, "v")
    rc = lib.gdnq_kv_append(
        d, r, None if r is None else _table(table, r, cur), _kv(kv, d, cur), qp, ldq, op, ldqo, kp, ldk, vp, ldv,
        _flat(pos, T, i32, cur, "pos"), _flat(slots, n, i32, cur, "slots"),
        _flat(cu_seqlens, n + 1, i32, cur, "cu_seqlens"), n, T, st)
    if rc:
        _check(rc)


def gdnq_attn_workspace(desc, kv, n) -> int:
    """Bytes of workspace that gdnq_attn_step needs."""
    out, d = ctypes.c_size_t(), _desc(desc)
    _check(lib.gdnq_attn_workspace(d, _kv(kv, d), n, ctypes.byref(out)))
    return out.value


def gdnq_attn_step(desc, kv, q, o, slots, n, workspace=None, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    io, _, i32 = _layer._types(d)
    kv = _kv(kv, d, cur)
    qp, ldq = _rows(q, n, d.H * d.d, io, cur, "q")
    op, ldo = _rows(o, n, d.H * d.d, io, cur, "o")
    ws, nb = _space(workspace, cur, lambda: gdnq_attn_workspace(d, kv, n))
    rc = lib.gdnq_attn_step(d, kv, qp, ldq, op, ldo, _flat(slots, n, i32, cur, "slots"), n, ws, nb, st)
    if rc:
        _check(rc)


def gdnq_kv_evict_workspace(desc, kv, budget, n) -> int:
    """Bytes of workspace that gdnq_kv_evict needs."""
    out, d = ctypes.c_size_t(), _desc(desc)
    _check(lib.gdnq_kv_evict_workspace(d, _kv(kv, d), budget, n, ctypes.byref(out)))
    return out.value


def gdnq_kv_evict(desc, kv, budget, sink, recent, slots, n, workspace=None, stream=None):
    d = _desc(desc)
    cur, st = _begin(stream)
    _, _, i32 = _layer._types(d)
    kv = _kv(kv, d, cur)
    ws, nb = _space(workspace, cur, lambda: gdnq_kv_evict_workspace(d, kv, budget, n))
    rc = lib.gdnq_kv_evict(d, kv, budget, sink, recent, _flat(slots, n, i32, cur, "slots"), n, ws, nb, st)
    if rc:
        _check(rc)
