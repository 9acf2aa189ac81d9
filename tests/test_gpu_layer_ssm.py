"""Selective state space scan (gdnq_ssm_prefill, gdnq_ssm_step) against the
recurrence in 64 bits, token by token (tests/_layer.py).

Bounds, with u = 2^-24 and each value's magnitude form (the recurrence on
absolute values, ym and Sm) as the measure:
  step: the decay a = e^{delta A} carries delta's relative error e_d times
  |delta A| and a few ulps, B (delta x)^T carries e_d, the sum over dk rows
  dk u; states then round once, outputs once to their type.
  prompts: chunks of 64 tokens or fewer.  An operand in two bf16 parts is off
  by at most 2^-16 of itself (2^-8 a part), in three by 2^-24.  An output
  takes C B^T and w x in two parts each and leaves out the product of their
  second parts: 3 2^-16.  Sums have at most dk and 64 terms, and a decay between
  two tokens of a chunk comes from a difference of running sums of at most K
  (the largest sum of |delta A| over 64 tokens), each off by at most 8 u K, so
  by a relative 16 u K; every chunk that a state passes through adds a
  rounding of its decay (8 u K + 4 u, at most K e^-K-weighted: 8 u) and of
  its sum."""
import numpy as np
import pytest

from tests import _layer as L
from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu


def _problem(seed, T, H, dk, dv, hk, io, n_slots, strong=False):
    """Host tensors of a call: rows in the io type, parameters in fp32."""
    torch = torch_cuda()
    r = np.random.default_rng(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    t = lambda *s, k=1.0: torch.from_numpy((r.standard_normal(s) * k).astype(np.float32)).to(dt)  # noqa: E731
    step = np.exp(r.uniform(np.log(1e-3), np.log(0.1), H))
    p = dict(x=t(T, H * dv), B=t(T, hk * dk, k=0.5), C=t(T, hk * dk, k=0.5), dt=t(T, H, k=0.5),
             A=-r.uniform(1, 16, H).astype(np.float32), D=r.standard_normal(H).astype(np.float32),
             dt_bias=(step + np.log(-np.expm1(-step))).astype(np.float32),
             S=(r.standard_normal((n_slots, H, dk, dv)) * 0.05).astype(np.float32))
    if strong:   # steps of about 3 and rates to 30: a chunk decays far below fp32's range
        p["dt_bias"] = np.full(H, 3.0, np.float32)
        p["A"] = -r.uniform(0, 30, H).astype(np.float32)
        p["A"][0] = 0.0
    return p


def _ref(p, first, end, S, H, dk, dv, hk, D=True, bias=True, **kw):
    f = lambda k: p[k][first:end].double().numpy()  # noqa: E731
    rep = lambda k: np.repeat(f(k).reshape(end - first, hk, dk), H // hk, axis=1)  # noqa: E731
    return L.ssm_rows(f("x").reshape(end - first, H, dv), rep("B"), rep("C"), f("dt"), p["A"].astype(np.float64),
                      p["D"].astype(np.float64) if D else None, p["dt_bias"].astype(np.float64) if bias else None,
                      S.astype(np.float64), **kw)


def _wide(t, off):
    torch = torch_cuda()
    w = torch.full((t.shape[0], t.shape[1] + 2 * off), 7.0, dtype=t.dtype, device="cuda")
    w[:, off:off + t.shape[1]] = t.cuda()
    return w[:, off:off + t.shape[1]], w


def _dev(p, off=0):
    torch = torch_cuda()
    d = {k: _wide(p[k], off)[0] for k in ("x", "B", "C", "dt")}
    d.update({k: torch.from_numpy(p[k]).cuda() for k in ("A", "D", "dt_bias", "S")})
    return d


STEPS = [("bf16", 1, 4, 128, 64, 1, 0), ("f32", 3, 4, 64, 64, 2, 0), ("bf16", 9, 6, 128, 128, 3, 8),
         ("f32", 5, 3, 64, 128, 3, 4), ("bf16", 4, 5, 128, 64, 1, 3), ("f32", 2, 8, 128, 128, 8, 1)]


@pytest.mark.parametrize("io,n,H,dk,dv,hk,off", STEPS)
def test_tokens(io, n, H, dk, dv, hk, off):
    torch = torch_cuda()
    g = lib()
    say("ssm tokens", io, n, H, dk, dv, hk, off)
    n_slots = n + 3
    p = _problem(n * 7 + H, n, H, dk, dv, hk, io, n_slots)
    d = _dev(p, off)
    slots = np.random.default_rng(n).permutation(n_slots)[:n].astype(np.int32)
    if n > 2:
        slots[1], slots[2] = -1, n_slots
    y, ywide = _wide(torch.full_like(p["x"], 7.0), off)
    desc = g.SsmDesc(H=H, dk=dk, dv=dv, hk=hk, io_dtype=g.IO_BF16 if io == "bf16" else g.IO_F32)
    g.gdnq_ssm_step(desc, d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], y, d["S"], n_slots,
                    torch.from_numpy(slots).cuda(), n)
    torch.cuda.synchronize()
    got, gS = y.double().cpu().numpy().reshape(n, H, dv), d["S"].double().cpu().numpy()
    want = p["S"].astype(np.float64)
    for i in range(n):
        if not 0 <= slots[i] < n_slots:
            assert (got[i] == 7).all()
            continue
        ref, S, ym, Sm, delta, v = _ref(p, i, i + 1, p["S"][slots[i]], H, dk, dv, hk)
        e = L.delta_bound(v[0]) * (1 + np.abs(delta[0] * p["A"])) + 8 * L.U
        assert not (np.abs(gS[slots[i]] - S) > Sm * e[:, None, None] + 2.0 ** -120).any()
        bound = ym[0] * (e + (dk + 8) * L.U)[:, None]
        assert not (np.abs(got[i] - ref[0]) > bound + (np.abs(ref[0]) + bound) * L.ROUND[io] + 2.0 ** -120).any()
        want[slots[i]] = gS[slots[i]]
    assert np.array_equal(want, gS)
    assert bool((ywide[:, :off] == 7).all()) and bool((ywide[:, off + H * dv:] == 7).all())


def test_tokens_options():
    """No softplus, clamped steps, no skip term, no bias, implicit slots."""
    torch = torch_cuda()
    g = lib()
    say("ssm token options")
    n, H, dk, dv = 3, 2, 64, 64
    p = _problem(3, n, H, dk, dv, 1, "f32", n)
    p["dt"] = torch.tensor([[0.5, -1.0], [1e-4, 0.02], [3.0, 0.05]])
    d = _dev(p)
    y = torch.empty_like(d["x"])
    desc = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1, io_dtype=g.IO_F32, flags=0, dt_min=0.001, dt_max=0.1)
    g.gdnq_ssm_step(desc, d["x"], d["B"], d["C"], d["dt"], d["A"], None, None, y, d["S"], n, None, n)
    torch.cuda.synchronize()
    for i in range(n):
        lo, hi = (float(np.float32(v)) for v in (0.001, 0.1))
        ref, S, ym, Sm, delta, v = _ref(p, i, i + 1, p["S"][i], H, dk, dv, 1, D=False, bias=False, sp=False, lo=lo,
                                        hi=hi)
        e = 16 * L.U * (1 + np.abs(delta[0] * p["A"]))
        assert not (np.abs(d["S"][i].double().cpu().numpy() - S) > Sm * e[:, None, None]).any()
        got = y[i].double().cpu().numpy().reshape(H, dv)
        assert not (np.abs(got - ref[0]) > ym[0] * (e + (dk + 8) * L.U)[:, None]).any()


PROMPTS = [  # H, dk, dv, hk, lens, tail, column offset, strong decays
    (2, 128, 64, 1, [1], 0, 0, False),
    (4, 128, 64, 1, [64, 63, 65, 1, 0, 2, 130], 7, 0, False),
    (4, 128, 128, 2, [33, 100, 0, 31, 32], 0, 0, False),
    (3, 64, 64, 3, [17, 200], 3, 0, False),
    (6, 64, 128, 2, [129, 5], 0, 8, False),
    (5, 128, 64, 1, [70, 128], 2, 3, False),
    (8, 128, 64, 1, [500, 3, 260], 0, 0, False),
    (4, 128, 64, 1, [150, 64, 9], 0, 0, True),
    (2, 64, 64, 1, [3] * 90 + [100, 0, 1], 5, 0, False),
    (2, 128, 64, 2, [2500], 0, 0, False),
    (1, 128, 128, 1, [700, 640], 0, 0, True),
    (7, 64, 128, 1, [1500, 90], 11, 0, False),
]


def _check_prompts(p, got, gS, slots, cont, cu, n_slots, H, dk, dv, hk):
    want, keep = p["S"].astype(np.float64), np.ones(got.shape[0], bool)
    for i in range(len(cu) - 1):
        lo, hi = cu[i], cu[i + 1]
        if hi == lo or not 0 <= slots[i] < n_slots:
            continue
        S0 = p["S"][slots[i]] * (cont is not None and cont[i])
        ref, S, ym, Sm, delta, v = _ref(p, lo, hi, S0, H, dk, dv, hk)
        m = hi - lo
        c = np.concatenate([np.zeros((1, H)), np.cumsum(np.abs(delta * p["A"]), 0)])
        K = max((c[min(t + 64, m)] - c[t]).max() for t in range(m))
        e_d = L.delta_bound(v).max() * (1 + min(K, 64))
        tau = e_d + (dk + 2 * 64 + 16 * K + 16 * (m // 32 + 1)) * L.U
        dS = np.abs(gS[slots[i]] - S) - Sm * (tau + 2.0 ** -24)
        assert not (dS > 2.0 ** -120).any(), (i, dS.max(), "state")
        b = ym * (tau + 3 * 2.0 ** -16 + dk * L.U)
        dy = np.abs(got[lo:hi] - ref) - (b + (np.abs(ref) + b) * L.ROUND["bf16"])
        assert not (dy > 2.0 ** -120).any(), (i, dy.max(), np.argwhere(dy > 0)[:4].tolist())
        want[slots[i]] = gS[slots[i]]
        keep[lo:hi] = False
    assert np.array_equal(want, gS), "a slot of no sequence changed"
    assert (got[keep] == 7).all(), "a row of no sequence changed"


@pytest.mark.parametrize("case", PROMPTS, ids=[f"H{c[0]}-{c[1]}x{c[2]}-hk{c[3]}-n{len(c[4])}-T{sum(c[4])}" for c in PROMPTS])
@pytest.mark.parametrize("mode", ["mixed", "new"])
def test_prompts(case, mode):
    torch = torch_cuda()
    g = lib()
    H, dk, dv, hk, lens, tail, off, strong = case
    say("ssm prompts", case, mode)
    n, T, n_slots = len(lens), sum(lens) + tail, len(lens) + 2
    p = _problem(T + H, T, H, dk, dv, hk, "bf16", n_slots, strong)
    d = _dev(p, off)
    r = np.random.default_rng(T)
    slots = r.permutation(n_slots)[:n].astype(np.int32)
    if n > 5:
        slots[1] = -1
    cont = r.integers(0, 2, n).astype(np.int32)
    cont[0] = 1
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    y, ywide = _wide(torch.full_like(p["x"], 7.0), off)
    desc = g.SsmDesc(H=H, dk=dk, dv=dv, hk=hk)
    nb = g.gdnq_ssm_workspace(desc, n, T)
    ws = torch.full((nb + 256,), 0x7F, dtype=torch.uint8, device="cuda")   # NaN-like bytes: nothing may rely on it
    g.gdnq_ssm_prefill(desc, d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], y, d["S"], n_slots,
                       up(slots), up(cont) if mode == "mixed" else None, up(cu), n, T, ws)
    torch.cuda.synchronize()
    assert bool((ws[nb:] == 0x7F).all()), "written behind the workspace"
    _check_prompts(p, y.double().cpu().numpy().reshape(T, H, dv), d["S"].double().cpu().numpy(), slots,
                   cont if mode == "mixed" else None, cu, n_slots, H, dk, dv, hk)
    assert bool((ywide[:, :off] == 7).all()) and bool((ywide[:, off + H * dv:] == 7).all())


# more than 384 tokens, many sequences: a workgroup takes several, the last of
# which may go on in another's (several short ones in a row, a cut just behind
# a start or before an end, empty ones between, hundreds of head blocks)
SHARED = [
    (64, 64, 64, 1, [3] * 60 + [900, 0, 1] + [2] * 30 + [65, 64, 0, 0, 127], 9, 0, False),
    (48, 128, 64, 1, [130, 120, 140, 1, 128, 64, 192, 500], 0, 0, True),
    (16, 128, 128, 2, [1, 1, 1, 1200, 1, 1, 300, 0, 450], 4, 8, False),
    (300, 64, 64, 300, [150, 60, 200], 1, 0, False),
    (9, 64, 128, 3, [385, 1, 1, 1, 1], 0, 2, False),
]


@pytest.mark.parametrize("case", SHARED, ids=[f"H{c[0]}-{c[1]}x{c[2]}-hk{c[3]}-n{len(c[4])}-T{sum(c[4])}" for c in SHARED])
@pytest.mark.parametrize("mode", ["mixed", "new"])
def test_prompts_that_share_workgroups(case, mode):
    test_prompts(case, mode)


def test_sequences_between_skipped_ones_of_long_calls():
    """Sequences with bounds before the first row, behind the last, or with a
    slot outside the pool are left out; those between them are whole."""
    torch = torch_cuda()
    g = lib()
    say("ssm long skips")
    H, dk, dv, T = 32, 64, 64, 1400
    cu = np.array([-3, 5, 300, 302, 500, 1290, 1390, 1401, 5000], np.int32)
    slots = np.array([0, 1, 2, 9, 4, 5, 6, 7], np.int32)
    cont = np.array([1, 1, 0, 1, 1, 0, 1, 1], np.int32)
    p = _problem(4, T, H, dk, dv, 1, "bf16", 8)
    d = _dev(p)
    y = torch.full_like(d["x"], 7.0)
    desc = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1)
    nb = g.gdnq_ssm_workspace(desc, 8, T)
    assert nb > 0
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    g.gdnq_ssm_prefill(desc, d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], y, d["S"], 8, up(slots),
                       up(cont), up(cu), 8, T, torch.full((nb,), 0x7F, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for i in (0, 6, 7):
        slots[i] = -1
    _check_prompts(p, y.double().cpu().numpy().reshape(T, H, dv), d["S"].double().cpu().numpy(), slots, cont, cu, 8,
                   H, dk, dv, 1)


@pytest.mark.parametrize("cu", [[0, 400, 1501], [-5, 400, 1000], [0, 2 ** 31 - 1, 1000], [1070, 960, 950],
                                [0, 900, -2 ** 31], [0, 900, 300], [-2 ** 31, 2 ** 31 - 1, 1500]])
def test_bounds_that_break_the_rules_of_long_calls(cu):
    torch = torch_cuda()
    g = lib()
    say("ssm long bounds", cu)
    H, dk, dv, T = 16, 64, 64, 1500
    p = _problem(1, T, H, dk, dv, 1, "bf16", 2)
    desc = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1)
    d = _dev(p)
    buf = torch.full((T + 128, H * dv), 3.0, dtype=torch.bfloat16, device="cuda")
    nb = g.gdnq_ssm_workspace(desc, 2, T)
    assert nb > 0
    ws = torch.zeros(nb + 64, dtype=torch.uint8, device="cuda")
    cont = torch.ones(2, dtype=torch.int32, device="cuda")
    g.gdnq_ssm_prefill(desc, d["x"], d["B"], d["C"], d["dt"], d["A"], None, None, buf[64:64 + T], d["S"], 2, None,
                       cont, torch.tensor(cu, dtype=torch.int32, device="cuda"), 2, T, ws)
    torch.cuda.synchronize()
    assert (buf[:64] == 3).all() and (buf[64 + T:] == 3).all()
    assert (ws[-64:] == 0).all()
    for i in range(2):
        if not 0 <= cu[i] < cu[i + 1] <= T:
            assert np.array_equal(d["S"][i].cpu().numpy(), p["S"][i])


def test_bounds_that_break_the_rules_touch_nothing_outside():
    torch = torch_cuda()
    g = lib()
    say("ssm bounds")
    H, dk, dv, T = 2, 64, 64, 200
    p = _problem(1, T, H, dk, dv, 1, "bf16", 2)
    desc = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1)
    for cu in ([0, 40, 201], [-5, 40, 100], [0, 2 ** 31 - 1, 100], [70, 60, 50], [0, 50, -2 ** 31]):
        d = _dev(p)
        buf = torch.full((T + 128, H * dv), 3.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros(g.gdnq_ssm_workspace(desc, 2, T) + 64, dtype=torch.uint8, device="cuda")
        g.gdnq_ssm_prefill(desc, d["x"], d["B"], d["C"], d["dt"], d["A"], None, None, buf[64:64 + T], d["S"], 2, None,
                           None, torch.tensor(cu, dtype=torch.int32, device="cuda"), 2, T, ws)
        torch.cuda.synchronize()
        assert (buf[:64] == 3).all() and (buf[64 + T:] == 3).all(), cu
        assert (ws[-64:] == 0).all(), cu
        for i in range(2):
            if not 0 <= cu[i] < cu[i + 1] <= T:
                assert np.array_equal(d["S"][i].cpu().numpy(), p["S"][i]), cu


@pytest.mark.parametrize("resets", [False, True])
def test_prompts_over_decays(resets):
    """Heads whose chunks decay by 2^-0 to 2^-5000, on every side of the
    kernel's two borders (2^-80 and 2^-160 over 64 tokens), evenly or by a few
    tokens that forget nearly everything before them."""
    torch = torch_cuda()
    g = lib()
    say("ssm decays", resets)
    bits = np.array([0, 1e-3, 20, 70, 79, 81, 100, 140, 158, 162, 400, 5000], np.float64)
    H, dk, dv, T = len(bits), 128, 64, 300
    p = _problem(77, T, H, dk, dv, 1, "bf16", 1)
    step = np.full((T, H), 0.25)
    if resets:
        step[:] = 1e-3
        step[np.random.default_rng(3).integers(0, T, 14)] = 4.0
    p["dt"] = torch.from_numpy(np.log(np.expm1(step)).astype(np.float32)).bfloat16()
    p["dt_bias"] = np.zeros(H, np.float32)
    per = 64 * 0.25 if not resets else 3 * 4.0
    p["A"] = (-bits * np.log(2.0) / per).astype(np.float32)
    d = _dev(p)
    y = torch.full_like(d["x"], 7.0)
    desc = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    nb = g.gdnq_ssm_workspace(desc, 1, T)
    g.gdnq_ssm_prefill(desc, d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], y, d["S"], 1, i32(0), i32(1),
                       i32(0, T), 1, T, torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None)
    torch.cuda.synchronize()
    _check_prompts(p, y.double().cpu().numpy().reshape(T, H, dv), d["S"].double().cpu().numpy(), [0], [1], [0, T], 1, H,
                   dk, dv, 1)
