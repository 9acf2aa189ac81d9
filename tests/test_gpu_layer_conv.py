"""Short causal convolution (gdnq_conv_prefill, gdnq_conv_step) against its
definition in 64 bits (tests/_layer.py).

Outputs: every element within the fp32 bound of the sum and the activation
plus one rounding to the output type.  States: equal bit for bit (they hold
the inputs themselves).  Memory around every output (other slots, rows of no
sequence, the columns between strided rows) must stay as it was."""
import numpy as np
import pytest

from tests import _layer as L
from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu

DT = {"bf16": "bfloat16", "f32": "float32"}


def _make(rng, shape, io, scale=1.0):
    torch = torch_cuda()
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(getattr(torch, DT[io]))
    return t


def _f64(t):
    return t.double().cpu().numpy()


def _strided(t, off, pad):
    """The same rows inside a wider buffer, `off` columns from its start, and that buffer."""
    torch = torch_cuda()
    wide = torch.full((t.shape[0], off + t.shape[1] + pad), 7.0, dtype=t.dtype)
    wide[:, off:off + t.shape[1]] = t
    wide = wide.cuda()
    return wide[:, off:off + t.shape[1]], wide


CASES = [
    # io, C, width, silu, bias, lens, T - sum(lens), column offset and padding of the rows
    ("bf16", 64, 4, True, True, [1], 0, 0, 0),
    ("f32", 4, 4, True, False, [2], 3, 0, 0),
    ("bf16", 520, 4, True, True, [0, 3, 1, 64, 2, 0, 65, 33], 5, 0, 0),
    ("bf16", 512, 3, False, True, [31, 32, 33, 7, 1], 0, 0, 0),
    ("f32", 260, 2, True, False, [100, 1, 0, 2], 1, 0, 0),
    ("bf16", 77, 4, True, True, [5, 40, 1, 0, 96], 2, 0, 0),
    ("f32", 131, 3, True, True, [64, 2, 70], 0, 0, 0),
    ("bf16", 128, 4, True, False, [50, 3, 80], 4, 8, 16),
    ("bf16", 128, 4, True, False, [50, 3, 80], 4, 3, 2),
    ("f32", 1024, 4, False, False, [300], 0, 4, 4),
    ("bf16", 1, 2, True, True, [17, 1], 0, 0, 0),
    ("bf16", 4096, 4, True, True, [700, 1, 0, 260], 9, 0, 0),
    ("bf16", 64, 4, True, True, [3] * 150 + [0, 1, 2, 40], 0, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-C{c[1]}-w{c[2]}-n{len(c[5])}-off{c[7]}" for c in CASES])
@pytest.mark.parametrize("mode", ["mixed", "new"])
def test_prompts(case, mode):
    torch = torch_cuda()
    g = lib()
    io, C, W, silu, bias, lens, tail, off, pad = case
    say("conv prompts", case, mode)
    rng = np.random.default_rng(C * 31 + W)
    n, total = len(lens), sum(lens)
    T, n_slots = total + tail, len(lens) + 3
    x = _make(rng, (T, C), io)
    xd, _ = _strided(x, off, pad)
    yd, ybuf = _strided(torch.full_like(x, 0.25), off, pad)
    ybefore = ybuf.clone()
    w = (rng.standard_normal((W, C)) / 2).astype(np.float32)
    b = rng.standard_normal(C).astype(np.float32) if bias else None
    state = _make(rng, (n_slots, W - 1, C), io)
    sd = state.cuda()
    slots = rng.permutation(n_slots)[:n].astype(np.int32)
    cont = rng.integers(0, 2, n).astype(np.int32)
    if n > 2:
        slots[1] = -1
        slots[2] = n_slots
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    up = lambda v: None if v is None else torch.from_numpy(v).cuda()  # noqa: E731
    desc = g.ConvDesc(C=C, width=W, io_dtype=g.IO_BF16 if io == "bf16" else g.IO_F32, flags=g.CONV_SILU if silu else 0)
    g.gdnq_conv_prefill(desc, xd, up(w), up(b), sd, n_slots, up(slots), up(cont) if mode == "mixed" else None,
                        up(cu), n, T, yd)
    torch.cuda.synchronize()
    want_state = state.clone()
    keep = torch.ones(ybuf.shape, dtype=torch.bool)
    for i, m in enumerate(lens):
        if m == 0 or not 0 <= slots[i] < n_slots:
            continue
        use = mode == "mixed" and cont[i]
        hist = _f64(state[slots[i]]) if use else np.zeros((W - 1, C))
        ref, new, err = L.conv_rows(_f64(x[cu[i]:cu[i + 1]]), hist, w.astype(np.float64),
                                    None if b is None else b.astype(np.float64), silu)
        got = _f64(yd[cu[i]:cu[i + 1]])
        bad = np.abs(got - ref) > err + (np.abs(ref) + err) * L.ROUND[io] + 2.0 ** -120
        assert not bad.any(), (i, bad.sum(), np.abs(got - ref).max())
        want_state[slots[i]] = torch.from_numpy(new).to(state.dtype)
        keep[cu[i]:cu[i + 1], off:off + C] = False
    assert torch.equal(sd.cpu(), want_state)
    assert torch.equal(ybuf.cpu()[keep], ybefore.cpu()[keep])


STEPS = [("bf16", 64, 4, 1), ("f32", 4, 2, 3), ("bf16", 77, 4, 5), ("bf16", 520, 3, 70), ("f32", 131, 3, 9),
         ("bf16", 4096, 4, 33), ("f32", 2052, 4, 12)]


@pytest.mark.parametrize("io,C,W,n", STEPS)
@pytest.mark.parametrize("off", [0, 8, 3])
def test_tokens(io, C, W, n, off):
    torch = torch_cuda()
    g = lib()
    say("conv tokens", io, C, W, n, off)
    rng = np.random.default_rng(C + n + off)
    n_slots = n + 4
    x = _make(rng, (n, C), io)
    xd, _ = _strided(x, off, off)
    yd, ybuf = _strided(torch.full_like(x, 0.25), off, off)
    ybefore = ybuf.clone()
    w = (rng.standard_normal((W, C)) / 2).astype(np.float32)
    b = rng.standard_normal(C).astype(np.float32)
    state = _make(rng, (n_slots, W - 1, C), io)
    sd = state.cuda()
    slots = rng.permutation(n_slots)[:n].astype(np.int32)
    if n > 2:
        slots[0], slots[2] = -1, n_slots + 5
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    desc = g.ConvDesc(C=C, width=W, io_dtype=g.IO_BF16 if io == "bf16" else g.IO_F32)
    g.gdnq_conv_step(desc, xd, up(w), up(b), sd, n_slots, up(slots), n, yd)
    torch.cuda.synchronize()
    want = state.clone()
    keep = torch.ones(ybuf.shape, dtype=torch.bool)
    for i in range(n):
        if not 0 <= slots[i] < n_slots:
            continue
        ref, new, err = L.conv_rows(_f64(x[i:i + 1]), _f64(state[slots[i]]), w.astype(np.float64),
                                    b.astype(np.float64), True)
        got = _f64(yd[i:i + 1])
        assert not (np.abs(got - ref) > err + (np.abs(ref) + err) * L.ROUND[io] + 2.0 ** -120).any(), i
        want[slots[i]] = torch.from_numpy(new).to(state.dtype)
        keep[i, off:off + C] = False
    assert torch.equal(sd.cpu(), want)
    assert torch.equal(ybuf.cpu()[keep], ybefore.cpu()[keep])


def test_prompt_then_tokens_equals_one_prompt():
    """A prompt cut anywhere and continued, by further prompts or token by
    token, gives the whole prompt's outputs and state bit for bit: every
    output is the same sequence of operations on the same inputs."""
    torch = torch_cuda()
    g = lib()
    say("conv prompt then tokens")
    rng = np.random.default_rng(5)
    C, W, T = 264, 4, 90
    x = _make(rng, (T, C), "bf16").cuda()
    w = torch.from_numpy(rng.standard_normal((W, C)).astype(np.float32)).cuda()
    desc = g.ConvDesc(C=C, width=W)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ones = i32(1)

    def prompt(s, y, lo, hi, cont):
        g.gdnq_conv_prefill(desc, x[lo:hi], w, None, s, 1, None, ones if cont else None, i32(0, hi - lo), 1, hi - lo,
                            y[lo:hi])

    whole_s, whole_y = torch.zeros(1, W - 1, C, dtype=x.dtype, device="cuda"), torch.zeros_like(x)
    prompt(whole_s, whole_y, 0, T, False)
    s, y = torch.zeros_like(whole_s), torch.zeros_like(x)
    for lo, hi in ((0, 1), (1, 3), (3, 40), (40, 80)):
        prompt(s, y, lo, hi, lo > 0)
    for t in range(80, T):
        g.gdnq_conv_step(desc, x[t:t + 1], w, None, s, 1, None, 1, y[t:t + 1])
    torch.cuda.synchronize()
    assert torch.equal(y, whole_y) and torch.equal(s, whole_s)


def test_bounds_that_break_the_rules_touch_nothing_outside():
    """Sequences whose bounds leave 0 <= start <= end <= T are skipped."""
    torch = torch_cuda()
    g = lib()
    say("conv bounds")
    C, T = 64, 100
    desc = g.ConvDesc(C=C)
    x = torch.ones(T, C, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(4, C, device="cuda")
    for cu in ([0, 40, 101], [-5, 40, 100], [0, 2 ** 31 - 1, 100], [70, 60, 50], [0, 50, -2 ** 31]):
        buf = torch.full((T + 64, C), 3.0, dtype=torch.bfloat16, device="cuda")
        state = torch.full((2, 3, C), 5.0, dtype=torch.bfloat16, device="cuda")
        g.gdnq_conv_prefill(desc, x, w, None, state, 2, None, None,
                            torch.tensor(cu, dtype=torch.int32, device="cuda"), 2, T, buf[32:32 + T])
        torch.cuda.synchronize()
        assert (buf[:32] == 3).all() and (buf[32 + T:] == 3).all(), cu
        for i in range(2):
            if not 0 <= cu[i] < cu[i + 1] <= T:
                assert (state[i] == 5).all(), cu
