"""Rotary positions (gdnq_rope) against their definition (tests/_attn.py):
every element within the fp32 bound plus one rounding to the output type;
memory around the rows stays as it was."""
import numpy as np
import pytest

from tests import _attn as L
from tests._attn_gpu import f64, io_of, rand, strided, up
from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu

SCALED = {"plain": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
          "turns": dict(base=5e5, factor=8.0, orig_len=8192.0, lo=1.0, hi=4.0),
          "index": dict(base=5e5, factor=16.0, orig_len=4096.0, lo=1.0, hi=32.0)}
CODES = dict(plain="ROPE_PLAIN", linear="ROPE_LINEAR", base="ROPE_BASE", turns="ROPE_RAMP_TURNS",
             index="ROPE_RAMP_INDEX")


def table_of(desc, kind="plain", **kw):
    g = lib()
    return g.gdnq_rope_table(desc, g.RopeFreqs(kind=getattr(g, CODES[kind]), **{**SCALED[kind], **kw})).cuda()


CASES = [
    # io, rows, H, d, rot, kind, amp, column offset, padding
    ("bf16", 1, 1, 2, 2, "plain", 1.0, 0, 0),
    ("bf16", 3, 18, 256, 64, "plain", 1.0, 0, 0),
    ("f32", 5, 3, 64, 64, "linear", 1.0, 0, 0),
    ("bf16", 70, 40, 128, 128, "index", 1.2772588, 0, 0),
    ("bf16", 67, 5, 128, 96, "turns", 1.0, 8, 8),
    ("f32", 33, 7, 80, 20, "base", 0.5, 4, 4),
    ("bf16", 9, 3, 66, 34, "plain", 1.0, 0, 0),
    ("bf16", 9, 3, 64, 32, "plain", 1.0, 1, 2),
    ("f32", 4, 1, 1024, 1024, "turns", 1.0, 0, 0),
    ("bf16", 1, 600, 64, 16, "plain", 1.0, 0, 0),
    ("f32", 1000, 2, 128, 126, "plain", 1.0, 0, 0),
    ("bf16", 2049, 3, 64, 64, "linear", 1.0, 0, 8),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:6])) + f"-off{c[7]}" for c in CASES])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("mode", ["out", "in place", "inverse"])
def test_rows(case, inter, mode):
    torch = torch_cuda()
    g = lib()
    io, rows, H, d, rot, kind, amp, off, pad = case
    say("rope", case, inter, mode)
    rng = np.random.default_rng(rows + 7 * d + rot)
    x = rand(rng, (rows, H * d), io)
    pos = rng.integers(0, 1 << 20, rows).astype(np.int32)
    pos[:5] = np.array([0, 1, 2 ** 31 - 1, -2 ** 31, -17], np.int32)[:rows]
    xd, xbuf = strided(x, off, pad)
    yd, ybuf = (xd, xbuf) if mode == "in place" else strided(torch.full_like(x, 0.25), off, pad + 16)
    before = ybuf.clone()
    inverse = mode == "inverse"
    desc = g.RopeDesc(d=d, rot=rot, io_dtype=io_of(io), amp=amp,
                      flags=(g.ROPE_INTERLEAVED if inter else 0) | (g.ROPE_INVERSE if inverse else 0))
    g.gdnq_rope(desc, table_of(desc, kind), xd, up(pos), yd, rows, H)
    torch.cuda.synchronize()
    ref, err = L.rotate(f64(x).reshape(rows, H, d), pos, L.theta(rot, kind, **SCALED[kind]), rot, inter, inverse,
                        float(np.float32(amp)))
    got = f64(yd).reshape(rows, H, d)
    assert np.array_equal(got[..., rot:], ref[..., rot:])          # copied as they are
    bad = np.abs(got - ref) > err + (np.abs(ref) + err) * L.ROUND[io]
    assert not bad.any(), (bad.sum(), np.abs(got - ref).max())
    ybuf[:, off:off + H * d] = before[:, off:off + H * d]
    assert torch.equal(ybuf, before)


def test_no_angle():
    """Position 0 leaves the values as they are, and frequencies divided apart turn apart."""
    torch = torch_cuda()
    g = lib()
    say("rope at 0")
    rng = np.random.default_rng(5)
    x = rand(rng, (6, 4 * 64), "f32").cuda()
    desc = g.RopeDesc(d=64, io_dtype=g.IO_F32)
    y = torch.empty_like(x)
    g.gdnq_rope(desc, table_of(desc), x, torch.zeros(6, dtype=torch.int32, device="cuda"), y, 6, 4)
    assert torch.equal(x, y)
    div = list(np.linspace(1, 40, 32))
    pos = np.arange(6, dtype=np.int32) * 1000
    g.gdnq_rope(desc, table_of(desc, divisors=div), x, up(pos), y, 6, 4)
    ref, err = L.rotate(f64(x).reshape(6, 4, 64), pos, L.theta(64, divisors=div), 64)
    assert not (np.abs(f64(y).reshape(6, 4, 64) - ref) > err + np.abs(ref) * L.U).any()


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(inter):
    """The inverse call is the gradient: against autograd of the formula in 64
    bits, and against differences of the forward call (which is linear, so that
    the difference over a step of one is its derivative)."""
    torch = torch_cuda()
    g = lib()
    say("rope gradient", inter)
    rng = np.random.default_rng(11)
    rows, H, d, rot = 7, 2, 64, 48
    flags = g.ROPE_INTERLEAVED if inter else 0
    fwd = g.RopeDesc(d=d, rot=rot, io_dtype=g.IO_F32, flags=flags, amp=1.25)
    bwd = g.RopeDesc(d=d, rot=rot, io_dtype=g.IO_F32, flags=flags | g.ROPE_INVERSE, amp=1.25)
    t, pos = table_of(fwd), rng.integers(0, 5000, rows).astype(np.int32)
    x, gy = rand(rng, (rows, H * d), "f32").cuda(), rand(rng, (rows, H * d), "f32").cuda()
    gx = torch.empty_like(x)
    g.gdnq_rope(bwd, t, gy, up(pos), gx, rows, H)
    a = torch.from_numpy((pos.astype(L.LD)[:, None] * L.theta(rot) % L.PI2).astype(np.float64))[:, None]
    leaf = x.double().cpu().reshape(rows, H, d).requires_grad_()
    u, w = (leaf[..., 0:rot:2], leaf[..., 1:rot:2]) if inter else (leaf[..., :rot // 2], leaf[..., rot // 2:rot])
    p, q = 1.25 * (u * a.cos() - w * a.sin()), 1.25 * (w * a.cos() + u * a.sin())
    y = torch.stack([p, q], -1).reshape(rows, H, rot) if inter else torch.cat([p, q], -1)
    torch.cat([y, leaf[..., rot:]], -1).backward(gy.double().cpu().reshape(rows, H, d))
    _, err = L.rotate(f64(gy).reshape(rows, H, d), pos, L.theta(rot), rot, inter, True, 1.25)
    ref = leaf.grad.numpy()
    assert not (np.abs(f64(gx).reshape(ref.shape) - ref) > err + np.abs(ref) * L.U).any()
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    g.gdnq_rope(fwd, t, x, up(pos), y0, rows, H)
    for c in (0, 1, rot // 2, rot - 1, d - 1, d + 3):
        e = x.clone()
        e[:, c] += 1.0
        g.gdnq_rope(fwd, t, e, up(pos), y1, rows, H)
        diff = (f64(y1) - f64(y0)) * f64(gy)
        # each call is within 10 u 1.25 (|a| + |b|) + u |y| of the formula, times the gradient over two values
        tol = 24 * L.U * 1.25 * (np.abs(f64(gy)).max() * 2 * (2 * np.abs(f64(e)).max() + 1)) * 2
        step = f64(e)[:, c] - f64(x)[:, c]
        assert np.abs(diff.sum(1) - f64(gx)[:, c] * step).max() < tol


LONG = [("bf16", 128, 128, 0), ("f32", 66, 34, 0), ("bf16", 128, 92, 3), ("bf16", 64, 20, 8)]


@pytest.mark.parametrize("io,d,rot,off", LONG)
@pytest.mark.parametrize("inter", [False, True])
def test_long_calls(io, d, rot, off, inter):
    """A call whose rows go past the caches gives what calls on its parts give, bit for bit."""
    torch = torch_cuda()
    g = lib()
    say("rope, long call", io, d, rot, off, inter)
    rows, H = 4200, 12 * 1024 // d
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d)
    x = torch.randn(rows, H * d + off, generator=gen, device="cuda")
    x = x.to(torch.bfloat16 if io == "bf16" else torch.float32)[:, off:]
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 977
    y, z = torch.zeros_like(x), torch.zeros_like(x)
    assert 2 * x.numel() * x.element_size() > 64 << 20
    desc = g.RopeDesc(d=d, rot=rot, io_dtype=io_of(io), flags=g.ROPE_INTERLEAVED if inter else 0)
    t = table_of(desc)
    g.gdnq_rope(desc, t, x, pos, y, rows, H)
    for lo in range(0, rows, 700):
        g.gdnq_rope(desc, t, x[lo:lo + 700], pos[lo:lo + 700], z[lo:lo + 700], 700, H)
    assert torch.equal(y, z) and not torch.equal(x, y)
