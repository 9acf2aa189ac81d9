"""Gates and norms of the layer operators at the ends of their arguments, in
fp32, where nothing hides behind an output's rounding.  u = 2^-24."""
import numpy as np
import pytest

from tests import _layer as L
from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu

# e^-|x| (exp2's ulp and the correction: 3 u), 1 + e (u), the reciprocal (2 u),
# the products with e and with the argument (u each)
GATE = 8 * L.U


def _z(rows, D):
    z = np.random.default_rng(rows).uniform(-80, 40, (rows, D)).astype(np.float32)
    z[0, :8] = [0, -0.0, 1e-30, -1e-30, 100, -100, 3.3e38, -3.3e38]
    return z


def _silu(z):
    e = np.exp(-np.abs(z))
    return z * np.where(z >= 0, 1, e) / (1 + e)


def test_convolution_gate_in_fp32():
    """Taps (0, 1): the sum is the token itself."""
    torch = torch_cuda()
    g = lib()
    say("conv gate fp32")
    n, C = 512, 64
    x = _z(n, C)
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    w = np.stack([np.zeros(C), np.ones(C)]).astype(np.float32)
    d = g.ConvDesc(C=C, width=2, io_dtype=g.IO_F32)
    ref = _silu(x.astype(np.float64))
    for step in (False, True):
        y, st = torch.empty(n, C, device="cuda"), torch.zeros(n, 1, C, device="cuda")
        if step:
            g.gdnq_conv_step(d, up(x), up(w), None, st, n, None, n, y)
        else:
            g.gdnq_conv_prefill(d, up(x), up(w), None, st, n, None, None,
                                torch.tensor([0, n], dtype=torch.int32, device="cuda"), 1, n, y)
        torch.cuda.synchronize()
        got = y.double().cpu().numpy()
        bad = ~(np.abs(got - ref) <= np.abs(ref) * GATE + 2.0 ** -120)
        assert not bad.any(), (step, bad.sum(), (np.abs(got - ref)[bad] / np.abs(ref[bad])).max() / L.U)


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("sig", [False, True])
def test_norm_gate_in_fp32(first, sig):
    """Groups of 16: 4 squares a thread and 4 in a tree of lanes (8 u, half
    of it in the root), 8 u of the mean, root, weight and products."""
    torch = torch_cuda()
    g = lib()
    say("norm gate fp32", first, sig)
    rows, D = 256, 16
    r = np.random.default_rng(1)
    x, z = r.standard_normal((rows, D)).astype(np.float32), _z(rows, D)
    z[0, 6:8] = 0.5   # z act(z) squared would leave fp32
    w = r.standard_normal(D).astype(np.float32)
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    y = torch.empty(rows, D, device="cuda")
    d = g.NormDesc(D=D, io_dtype=g.IO_F32, eps=1e-5,
                   flags=(g.NORM_GATE_SIGMOID if sig else 0) | (g.NORM_GATE_FIRST if first else 0))
    g.gdnq_norm_gated(d, up(x), up(z), up(w), y, rows)
    torch.cuda.synchronize()
    x64, z64 = x.astype(np.float64), z.astype(np.float64)
    act = _silu(z64)
    if sig:
        e = np.exp(-np.abs(z64))
        act = np.where(z64 >= 0, 1, e) / (1 + e)
    u = x64 * act if first else x64
    ref = u * L.rms_rows(u, 1e-5) * w.astype(np.float64)
    ref = ref if first else ref * act
    got = y.double().cpu().numpy()
    rel = 12 * L.U + (2 * (GATE + L.U) if first else GATE)
    bad = ~(np.abs(got - ref) <= np.abs(ref) * rel + 2.0 ** -120)
    assert not bad.any(), (bad.sum(), (np.abs(got - ref)[bad] / np.abs(ref[bad])).max() / L.U)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [1e-40, 1e-38, 2e-45])
def test_smallest_eps(io, eps):
    """eps below fp32's normal numbers: rows of zeros give zeros, rows whose
    mean square is as small their own root.  Such an argument is a multiple of
    2^-149 and off by at most 4 of them (the mean's product and its sum with
    eps, half each, and 16 squares or sums of their own)."""
    torch = torch_cuda()
    g = lib()
    say("smallest eps", io, eps)
    D = 64
    r = np.random.default_rng(2)
    x = r.standard_normal((5, D)).astype(np.float32)
    x[0], x[1], x[2], x[3] = 0, x[1] * 2.0 ** -63, x[2] * 2.0 ** -66, x[3] * 2.0 ** -100
    x = torch.from_numpy(x).to(torch.bfloat16 if io == "bf16" else torch.float32)
    w = torch.ones(D, device="cuda")
    d = g.NormDesc(D=D, io_dtype=g.IO_BF16 if io == "bf16" else g.IO_F32, eps=eps)
    eps = float(np.float32(eps))
    y, y2, ro = (torch.full((5, D), 7.0, dtype=x.dtype, device="cuda") for _ in range(3))
    g.gdnq_norm_gated(d, x.cuda(), None, w, y, 5)
    g.gdnq_norm_residual(d, x.cuda(), w, 1.0, torch.zeros_like(x).cuda(), ro, w, y2, 5)
    torch.cuda.synchronize()
    u = x.double().numpy()
    arg = (u * u).mean(-1, keepdims=True) + eps
    tiny = 80 * 2.0 ** -149   # 64 squares of half a 2^-149 each, twice over
    ref = u / np.sqrt(arg)
    off = 0.5 * (2.0 * tiny / D + 2.0 ** -148) / arg
    got = y.double().cpu().numpy()
    assert np.isfinite(got).all() and np.isfinite(y2.double().cpu().numpy()).all()
    assert (got[0] == 0).all() and (y2[0] == 0).all()
    ok = off[:, 0] < 0.25   # beyond, the argument has no digits: eps = 2^-149 alone is one unit (row 0: zeros, above)
    assert ok[4]
    bad = np.abs(got - ref)[ok] > (np.abs(ref) * (40 * L.U + 2 * off + L.ROUND[io]))[ok]
    assert not bad.any(), np.abs(got / np.where(ref == 0, 1, ref) - 1).max(1)
