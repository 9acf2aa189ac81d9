"""Norms around a block (gdnq_norm_gated, gdnq_norm_residual) against their
definitions in 64 bits.

Bounds (u = 2^-24): a thread adds up to 32 squares, then at most 10 partial
sums are added in a tree of lanes and up to 16 in a row, so the sum of
squares of exact values is within (32 + 10 + 16) u of itself, its root within
half of that; the mean, eps, the reciprocal root (2 u), the weight's sum and
the products add 8 u: REL = 40 u.  A gate's relative error is at most
(2 |z| + 8) u, and values off by a relative e move their own norm by at most
the largest e.  Outputs add one rounding to their type."""
import numpy as np
import pytest

from tests import _layer as L
from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu

REL = 40 * L.U


def _t(rng, shape, io, scale=1.0):
    torch = torch_cuda()
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(
        torch.bfloat16 if io == "bf16" else torch.float32)


def _inside(t, off):
    torch = torch_cuda()
    wide = torch.full((t.shape[0], t.shape[1] + 2 * off), 7.0, dtype=t.dtype, device="cuda")
    wide[:, off:off + t.shape[1]] = t.cuda()
    return wide[:, off:off + t.shape[1]], wide


def _edges_kept(wide, off, width):
    return bool((wide[:, :off] == 7).all()) and bool((wide[:, off + width:] == 7).all())


GATED = [  # io, rows, D, group, offset of the rows
    ("bf16", 1, 8, 8, 0), ("f32", 3, 1, 1, 0), ("bf16", 7, 128, 128, 0), ("bf16", 5, 1024, 128, 0),
    ("f32", 9, 512, 64, 0), ("bf16", 3, 768, 256, 8), ("bf16", 2, 2048, 512, 0), ("bf16", 4, 1000, 1000, 0),
    ("bf16", 3, 777, 777, 0), ("f32", 2, 999, 333, 0), ("bf16", 5, 384, 128, 3), ("bf16", 2, 4096, 4096, 0),
    ("f32", 2, 4096, 4096, 0), ("bf16", 2, 8200, 8200, 0), ("f32", 1, 16388, 16388, 0), ("bf16", 1, 32768, 32768, 0),
    ("f32", 1, 32768, 32768, 0), ("bf16", 1, 32767, 32767, 0), ("f32", 1, 20001, 20001, 0), ("bf16", 1, 9999, 9999, 0),
    ("f32", 33, 96, 24, 0), ("bf16", 1, 6144, 2048, 0), ("f32", 2, 1536, 1536, 4), ("bf16", 3, 60, 20, 0),
]


@pytest.mark.parametrize("case", GATED, ids=[f"{c[0]}-{c[1]}x{c[2]}-g{c[3]}-o{c[4]}" for c in GATED])
@pytest.mark.parametrize("first,sig,shared,gate", [(False, False, True, True), (True, False, False, True),
                                                   (False, True, False, True), (True, True, True, True),
                                                   (False, False, False, False)])
def test_gated(case, first, sig, shared, gate):
    torch = torch_cuda()
    g = lib()
    io, rows, D, group, off = case
    say("gated norm", case, first, sig, shared, gate)
    rng = np.random.default_rng(D + rows)
    x, z = _t(rng, (rows, D), io, 2.0), _t(rng, (rows, D), io, 3.0)
    x[0, :group] = 0     # a row of zeros has an output of zeros
    w = rng.standard_normal(group if shared else D).astype(np.float32)
    xd, _ = _inside(x, off)
    zd, _ = _inside(z, off)
    yd, wide = _inside(torch.full_like(x, 7.0), off)
    flags = (g.NORM_GATE_SIGMOID if sig else 0) | (g.NORM_GATE_FIRST if first else 0)
    flags |= g.NORM_GROUP_WEIGHT if shared else 0
    d = g.NormDesc(D=D, group=group, io_dtype=g.IO_BF16 if io == "bf16" else g.IO_F32, flags=flags, eps=1e-5,
                   w_offset=1.0 if sig else 0.0)
    g.gdnq_norm_gated(d, xd, zd if gate else None, torch.from_numpy(w).cuda(), yd, rows)
    torch.cuda.synchronize()
    x64, z64 = (t.double().numpy().reshape(rows, D // group, group) for t in (x, z))
    s = L.sigmoid(z64)
    act = (s if sig else z64 * s) if gate else np.ones_like(z64)
    w64 = (w.astype(np.float64) if shared else w.astype(np.float64).reshape(D // group, group)) + d.w_offset
    u = x64 * act if first else x64
    ref = u * L.rms_rows(u, 1e-5) * w64
    ref = ref if first else ref * act
    rel = REL + (2 * ((2 * np.abs(z64) + 8) * L.U).max(-1, keepdims=True) if gate else 0)
    got = yd.double().cpu().numpy().reshape(ref.shape)
    bad = np.abs(got - ref) > np.abs(ref) * (rel + L.ROUND[io]) + 2.0 ** -120
    assert not bad.any(), (bad.sum(), np.abs(got - ref).max())
    assert _edges_kept(wide, off, D)


RES = [("bf16", 1, 8, 0), ("f32", 1, 2048, 0), ("bf16", 3, 4096, 0), ("bf16", 5, 777, 0), ("f32", 2, 333, 0),
       ("bf16", 4, 128, 8), ("bf16", 4, 128, 3), ("f32", 17, 64, 4), ("bf16", 2, 8192, 0), ("bf16", 1, 32768, 0),
       ("f32", 1, 32764, 0), ("bf16", 1, 30001, 0), ("f32", 3, 1, 0)]


@pytest.mark.parametrize("case", RES, ids=[f"{c[0]}-{c[1]}x{c[2]}-o{c[3]}" for c in RES])
@pytest.mark.parametrize("r32", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_residual(case, r32, post, inplace):
    torch = torch_cuda()
    g = lib()
    io, rows, D, off = case
    say("residual norm", case, r32, post, inplace)
    rng = np.random.default_rng(D * 3 + rows)
    scale = np.float32(0.37)
    rio = "f32" if r32 else io
    x, res = _t(rng, (rows, D), io), _t(rng, (rows, D), rio, 3.0)
    w, pw = rng.standard_normal(D).astype(np.float32), rng.standard_normal(D).astype(np.float32)
    xd, _ = _inside(x, off)
    rd, rwide = _inside(res, off)
    od, owide = (rd, rwide) if inplace else _inside(torch.full_like(res, 7.0), off)
    yd, ywide = _inside(torch.full_like(x, 7.0), off)
    d = g.NormDesc(D=D, io_dtype=g.IO_BF16 if io == "bf16" else g.IO_F32, flags=g.NORM_RES_F32 if r32 else 0,
                   eps=1e-6, w_offset=1.0)
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    g.gdnq_norm_residual(d, xd, up(pw) if post else None, float(scale), rd, od, up(w), yd, rows)
    torch.cuda.synchronize()
    p = x.double().numpy()
    perr = np.zeros_like(p)
    if post:
        p = p * L.rms_rows(p, 1e-6) * (1.0 + pw.astype(np.float64))
        perr = np.abs(p) * REL
    s64, r64 = float(scale), res.double().numpy()
    r = r64 + s64 * p
    rerr = s64 * perr + np.abs(r) * L.U
    got = od.double().cpu().numpy()
    assert not (np.abs(got - r) > rerr + (np.abs(r) + rerr) * L.ROUND[rio] + 2.0 ** -120).any()
    ref = r * L.rms_rows(r, 1e-6) * (1.0 + w.astype(np.float64))
    move = np.sqrt((rerr ** 2).sum(-1, keepdims=True) / np.maximum((r ** 2).sum(-1, keepdims=True), 1e-300))
    yerr = np.abs(L.rms_rows(r, 1e-6) * (1.0 + w.astype(np.float64))) * rerr + np.abs(ref) * (REL + 1.01 * move)
    gy = yd.double().cpu().numpy()
    bad = np.abs(gy - ref) > 1.01 * yerr + np.abs(ref) * L.ROUND[io] + 2.0 ** -120
    assert not bad.any(), (bad.sum(), np.abs(gy - ref).max())
    assert _edges_kept(ywide, off, D) and _edges_kept(owide, off, D)
    if not inplace:
        assert torch.equal(rd.cpu(), res)
    # the sum alone
    o2, _ = _inside(torch.full_like(res, 7.0), off)
    if not inplace:
        g.gdnq_norm_residual(d, xd, up(pw) if post else None, float(scale), rd, o2, None, None, rows)
        torch.cuda.synchronize()
        assert torch.equal(o2, od)
