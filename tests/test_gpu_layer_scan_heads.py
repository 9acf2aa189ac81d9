"""The scan's prompts (gdnq_ssm_prefill) head by head: bounds from each head's
own decays, neighbours in chunks that forget much, states in norm, the
descriptor's options, magnitudes at the ends of the stated range.  Bounds as
in test_gpu_layer_ssm.py unless a test derives its own, u = 2^-24."""
import numpy as np
import pytest

from tests import _layer as L
from tests._gpu import lib, say, torch_cuda
from tests.test_gpu_layer_ssm import _dev, _problem

pytestmark = pytest.mark.gpu


def _call(p, lens, H, dk, dv, hk, *, tail=0, cont=None, D=True, bias=True, **desc):
    """Runs a packed call; y and the states in 64 bits."""
    torch = torch_cuda()
    g = lib()
    n, T = len(lens), sum(lens) + tail
    d = _dev(p)
    y = torch.full_like(d["x"], 7.0)
    de = g.SsmDesc(H=H, dk=dk, dv=dv, hk=hk, **desc)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    nb = g.gdnq_ssm_workspace(de, n, T)
    ws = torch.full((nb,), 0x7F, dtype=torch.uint8, device="cuda") if nb else None
    g.gdnq_ssm_prefill(de, d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"] if D else None,
                       d["dt_bias"] if bias else None, y, d["S"], n, None, None if cont is None else i32(cont),
                       i32([0] + list(np.cumsum(lens))), n, T, ws)
    torch.cuda.synchronize()
    return y.double().cpu().numpy().reshape(T, H, dv), d["S"].double().cpu().numpy()


def _ref(p, first, end, S, H, dk, dv, hk, D=True, bias=True, **kw):
    f = lambda k: p[k][first:end].double().numpy()  # noqa: E731
    rep = lambda k: np.repeat(f(k).reshape(end - first, hk, dk), H // hk, axis=1)  # noqa: E731
    return L.ssm_rows(f("x").reshape(end - first, H, dv), rep("B"), rep("C"), f("dt"), p["A"].astype(np.float64),
                      p["D"].astype(np.float64) if D else None, p["dt_bias"].astype(np.float64) if bias else None,
                      S.astype(np.float64), **kw)


def _check(p, got, gS, lens, cont, H, dk, dv, hk, low=2.0 ** -120, exact_delta=False, **kw):
    """Every head within the bound of its own decays.  The exponents of a
    chunk that decays past 2^-160 are exact to 64 u; the running sums of the
    others reach 111 = 160 log 2 at most."""
    at = 0
    for i, m in enumerate(lens):
        end = at + m
        if m:
            ref, S, ym, Sm, delta, v = _ref(p, at, end, p["S"][i] * (cont is not None and cont[i]), H, dk, dv, hk, **kw)
            c = np.concatenate([np.zeros((1, H)), np.cumsum(np.abs(delta * p["A"]), 0)])
            K = np.max([c[min(t + 64, m)] - c[t] for t in range(m)], 0)
            e_d = 2 * L.U if exact_delta else L.delta_bound(v).max(0)
            tau = e_d * (1 + np.minimum(K, 64)) + (dk + 128 + 16 * np.minimum(K, 111) + 64 + 16 * (m // 32 + 1)) * L.U
            bad = np.abs(gS[i] - S) > Sm * (tau + 2.0 ** -24)[:, None, None] + low
            assert not bad.any(), (i, "state", np.unique(np.argwhere(bad)[:, 0]))
            b = ym * (tau + 3 * 2.0 ** -16 + dk * L.U)[None, :, None] + low
            bad = np.abs(got[at:end] - ref) > b + (np.abs(ref) + b) * L.ROUND["bf16"]
            assert not bad.any(), (i, "y", np.unique(np.argwhere(bad)[:, 1]))
        at = end
    assert (got[at:] == 7).all()


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_neighbours_between_tokens_that_forget(dk, dv):
    """Triples of a token that forgets everything before it (x = 0) and two
    with x of opposite signs, all B and C positive: the last token's output is
    C B delta x (e^{delta A} - 1), far below its two terms, so it shows how
    exact the decay between neighbours is, wherever in a chunk they stand.
    Steps are given (no softplus), so a term is off by its operands (3 2^-16),
    the two sums ((dk + 64) u), the exponent (64 u and its roundings: 8 u) and
    a few roundings (8 u)."""
    torch = torch_cuda()
    say("scan neighbours", dk, dv)
    H, T = 6, 640
    p = _problem(5, T, H, dk, dv, 1, "bf16", 1)
    for k in ("B", "C"):
        p[k] = p[k].abs()
    x = p["x"].reshape(T, H, dv)
    x[0::3] = 0
    x[2::3] = -x[1::3][:len(x[2::3])]
    dt = torch.full((T, H), 2.0 ** -9)
    dt[0::3] = torch.tensor([1.0, 5.0, 20.0, 77.0, 120.0, 200.0])
    p["dt"] = dt.bfloat16()
    p["A"] = -np.array([11.0, 15.0, 3.0, 2.0, 1.7, 1.1], np.float32)
    got, gS = _call(p, [T], H, dk, dv, 1, D=False, bias=False, cont=[1], flags=0)
    ref, S, ym, Sm, _, _ = _ref(p, 0, T, p["S"][0], H, dk, dv, 1, D=False, bias=False, sp=False)
    b = ym * (3 * 2.0 ** -16 + (dk + 144) * L.U)
    bad = np.abs(got - ref) > b + (np.abs(ref) + b) * L.ROUND["bf16"] + 2.0 ** -120
    assert not bad.any(), (bad.sum(), (np.abs(got - ref) / np.maximum(ym, 1e-30)).max())
    assert not (np.abs(gS[0] - S) > Sm * ((dk + 144) * L.U) + 2.0 ** -120).any()


@pytest.mark.parametrize("T", [64, 100, 640])
def test_states_in_norm(T):
    """||S - ref|| / ||ref|| per head.  Steps are given and every value is
    random, so errors add in quadrature: a weight (2 u), its product with x
    and its three parts (u each) and 12 additions a chunk, each half an ulp of
    the sum so far, stay below 8 u up to two chunks; ten chunks, with the
    roundings of their decays on one side, below 16 u.  (w x in two bf16 parts
    is off by 28 u or more, an exponent rounded at 2^6 by 13 u.)  In each chunk one
    token, with x = 0, decays by the head's bits, on every side of the
    kernel's borders."""
    torch = torch_cuda()
    say("scan states in norm", T)
    bits = np.array([0, 20, 79, 82, 110, 157, 163, 400], np.float64)
    H, dk, dv = len(bits), 128, 64
    p = _problem(T, T, H, dk, dv, 1, "bf16", 1)
    r = np.random.default_rng(T)
    dt = r.uniform(1e-3, 2e-2, (T, H)).astype(np.float32)
    p["A"] = np.full(H, -1.0, np.float32)
    p["A"][0] = 0.0
    x = p["x"].reshape(T, H, dv)
    for t in range(9, T, 64):
        dt[t] = np.maximum(bits * np.log(2.0), 1.0)
        x[t] = 0
    p["dt"] = torch.from_numpy(dt).bfloat16()
    _, gS = _call(p, [T], H, dk, dv, 1, D=False, bias=False, cont=[1], flags=0)
    _, S, _, _, _, _ = _ref(p, 0, T, p["S"][0], H, dk, dv, 1, D=False, bias=False, sp=False)
    off = np.sqrt(((gS[0] - S) ** 2).sum((1, 2)) / (S ** 2).sum((1, 2))) / L.U
    assert off.max() < (8 if T <= 128 else 16), off


@pytest.mark.parametrize("lens", [[130], [500, 60]])
def test_steps_of_the_largest_and_lowest_value(lens):
    """dt at the ends of its type: a step of dt_max, or of dt_min (a token
    that leaves the state as it was, where that is 0)."""
    torch = torch_cuda()
    say("scan dt ends", lens)
    H, dk, dv, T = 2, 64, 64, sum(lens)
    p = _problem(T, T, H, dk, dv, 1, "bf16", len(lens))
    top = torch.finfo(torch.bfloat16).max
    p["dt"][3::7] = top
    p["dt"][5::7] = -top
    p["dt_bias"] = np.zeros(H, np.float32)
    kw = dict(lo=0.0, hi=0.25)
    got, gS = _call(p, lens, H, dk, dv, 1, cont=[1] * len(lens), dt_min=0.0, dt_max=0.25)
    q = dict(p, dt=p["dt"].float().clamp(-100, 40))   # the same steps: softplus is 0 and above dt_max beyond
    _check(q, got, gS, lens, [1] * len(lens), H, dk, dv, 1, **kw)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_tokens_with_steps_of_the_largest_and_lowest_value(io):
    torch = torch_cuda()
    g = lib()
    say("scan token dt ends", io)
    H, dk, dv, n = 2, 64, 64, 4
    p = _problem(n, n, H, dk, dv, 1, io, n)
    top = torch.finfo(p["dt"].dtype).max
    p["dt"][1], p["dt"][2] = top, -top
    p["dt_bias"] = np.zeros(H, np.float32)
    d = _dev(p)
    y = torch.empty_like(d["x"])
    g.gdnq_ssm_step(g.SsmDesc(H=H, dk=dk, dv=dv, hk=1, io_dtype=g.IO_BF16 if io == "bf16" else g.IO_F32, dt_max=0.25),
                    d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], y, d["S"], n, None, n)
    torch.cuda.synchronize()
    q = dict(p, dt=p["dt"].float().clamp(-100, 40))
    for i in range(n):
        ref, S, ym, Sm, delta, v = _ref(q, i, i + 1, p["S"][i], H, dk, dv, 1, lo=0.0, hi=0.25)
        e = L.delta_bound(v[0]) * (1 + np.abs(delta[0] * p["A"])) + 8 * L.U
        assert not (np.abs(d["S"][i].double().cpu().numpy() - S) > Sm * e[:, None, None] + 2.0 ** -120).any()
        b = ym[0] * (e + (dk + 8) * L.U)[:, None]
        got = y[i].double().cpu().numpy().reshape(H, dv)
        assert not (np.abs(got - ref[0]) > b + (np.abs(ref[0]) + b) * L.ROUND[io] + 2.0 ** -120).any()


def _packed(g, T, lens, n, H=64, dk=128, dv=64):
    """A call of `lens` in n sequences (the rest empty) over T rows, as a closure."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(1)
    t = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    de = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1).c()
    x, B, C, dt = t(T, H * dv), t(T, dk), t(T, dk), t(T, H)
    A = -torch.rand(H, generator=gen, device="cuda") - 1
    S = torch.zeros(n, H, dk, dv, device="cuda")
    cu = torch.full((n + 1,), sum(lens), dtype=torch.int32, device="cuda")
    cu[:len(lens) + 1] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    ws = torch.empty(max(1, g.gdnq_ssm_workspace(de, n, T)), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    return lambda: g.gdnq_ssm_prefill(de, x, B, C, dt, A, None, None, y, S, n, None, None, cu, n, T, ws)


def _time(f):
    torch = torch_cuda()
    best = 1e9
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        f()
        a.record()
        for _ in range(5):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 5)
    return best


@pytest.mark.parametrize("T,lens,n", [(4096, [4096], 512), (4096, [3000, 1096], 256), (16384, [2048], 64),
                                      (16384, [2048], 1)])
def test_padded_batches_take_no_longer(T, lens, n):
    """Empty sequences behind the last and rows of none (a batch padded to
    the sizes of a captured graph) leave the work spread over the card."""
    g = lib()
    say("scan padded", T, lens, n)
    plain, padded = _time(_packed(g, sum(lens), lens, len(lens))), _time(_packed(g, T, lens, n))
    print(f"{plain * 1e3:.1f} us, padded {padded * 1e3:.1f} us")
    assert padded < 2 * plain


@pytest.mark.parametrize("lens,tail", [([700, 0, 33] + [0] * 60, 0), ([0] * 40 + [450] + [0] * 300, 900), ([129, 500], 3000),
                                       ([600], 2000), ([0] * 5, 1000), ([5] + [0] * 70, 600)])
def test_padded_batches(lens, tail):
    say("scan padded values", len(lens), tail)
    H, dk, dv, T = 8, 64, 64, sum(lens) + tail
    p = _problem(T, T, H, dk, dv, 2, "bf16", len(lens))
    cont = [i % 2 for i in range(len(lens))]
    got, gS = _call(p, lens, H, dk, dv, 2, tail=tail, cont=cont)
    _check(p, got, gS, lens, cont, H, dk, dv, 2)
    for i, m in enumerate(lens):
        if m == 0:
            assert np.array_equal(gS[i], p["S"][i].astype(np.float64))


@pytest.mark.parametrize("kind", ["even", "resets", "strong"])
def test_each_head_by_its_own_decays(kind):
    torch = torch_cuda()
    say("scan heads", kind)
    bits = np.array([0, 1e-3, 20, 70, 79, 81, 100, 140, 158, 162, 400, 5000], np.float64)
    H, dk, dv, lens = len(bits), 128, 64, [300, 0, 1, 520]
    T = sum(lens)
    p = _problem(78, T, H, dk, dv, 2, "bf16", len(lens), kind == "strong")
    if kind != "strong":
        step = np.full((T, H), 0.25)
        if kind == "resets":
            step[:] = 1e-3
            step[np.random.default_rng(3).integers(0, T, 3 * T // 64)] = 4.0
        p["dt"] = torch.from_numpy(np.log(np.expm1(step)).astype(np.float32)).bfloat16()
        p["dt_bias"] = np.zeros(H, np.float32)
        p["A"] = (-bits * np.log(2.0) / (16.0 if kind == "even" else 12.0)).astype(np.float32)
    cont = [1, 0, 1, 1]
    got, gS = _call(p, lens, H, dk, dv, 2, cont=cont)
    _check(p, got, gS, lens, cont, H, dk, dv, 2)


@pytest.mark.parametrize("lens", [[100, 7], [700, 90]])
@pytest.mark.parametrize("sp,D,bias", [(False, True, False), (True, False, True), (False, False, True), (True, True, False)])
def test_options(lens, sp, D, bias):
    """No softplus, clamped steps, no skip term, no bias."""
    g = lib()
    say("scan options", lens, sp, D, bias)
    H, dk, dv, T = 4, 64, 128, sum(lens)
    p = _problem(T, T, H, dk, dv, 2, "bf16", len(lens))
    lo, hi = np.float32(0.004), np.float32(0.3)
    if not sp:
        p["dt"] = (p["dt"].float() * 0.3).bfloat16()   # about half of them below zero
    got, gS = _call(p, lens, H, dk, dv, 2, D=D, bias=bias, cont=[1, 1], flags=g.SSM_SOFTPLUS if sp else 0,
                    dt_min=float(lo), dt_max=float(hi))
    _check(p, got, gS, lens, [1, 1], H, dk, dv, 2, D=D, bias=bias, sp=sp, lo=float(lo), hi=float(hi))


@pytest.mark.parametrize("power", [-30, 0, 38])
def test_magnitudes(power):
    """States and inputs at the ends of the stated range, over decays up to
    the kernel's borders.  What an output loses below it: parts of S 2^cs and
    of w x under 2^-126, whose row's factor is 2^80 at most."""
    torch = torch_cuda()
    say("scan magnitudes", power)
    bits = np.array([0, 20, 70, 79, 82, 110, 150, 158, 163, 900], np.float64)
    H, dk, dv, lens = len(bits), 128, 64, [200, 450]
    T = sum(lens)
    p = _problem(9, T, H, dk, dv, 1, "bf16", 2)
    p["x"] = p["x"] * 2.0 ** power
    p["S"] = (p["S"] * 2.0 ** power).astype(np.float32)
    p["dt"] = torch.full((T, H), 0.25).bfloat16()
    p["A"] = (-bits * np.log(2.0) / 16.0).astype(np.float32)
    got, gS = _call(p, lens, H, dk, dv, 1, bias=False, cont=[1, 1], flags=0)
    C = p["C"].double().abs().sum(1).max().item()
    CB = 64 * (p["C"].double() @ p["B"].double().T).abs().max().item()
    _check(p, got, gS, lens, [1, 1], H, dk, dv, 1, low=2.0 ** -46 * (C + CB), exact_delta=True, bias=False, sp=False)


def test_one_graph_for_batches_of_many_sizes():
    """A call captured at its largest size, replayed over other bounds: each
    replay equals the eager call on the same bounds, bit for bit."""
    torch = torch_cuda()
    g = lib()
    say("scan graph of padded batches")
    H, dk, dv, n, T = 16, 128, 64, 24, 3000
    p = _problem(6, T, H, dk, dv, 1, "bf16", n)
    d = _dev(p)
    S0, y = d["S"].clone(), torch.zeros_like(d["x"])
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cont = torch.ones(n, dtype=torch.int32, device="cuda")
    de = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1)
    ws = torch.empty(g.gdnq_ssm_workspace(de, n, T), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        g.gdnq_ssm_prefill(de, d["x"], d["B"], d["C"], d["dt"], d["A"], d["D"], d["dt_bias"], y, d["S"], n, None, cont, cu,
                           n, T, ws, stream=stream)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([T], [1] * n, [700, 0, 800, 1], [0, 0, 5], [], [125] * n, [2999] + [0] * 10 + [1], [400] * 7):
        bounds = np.full(n + 1, sum(lens))
        bounds[:len(lens) + 1] = np.concatenate([[0], np.cumsum(lens)])
        cu.copy_(torch.from_numpy(bounds.astype(np.int32)))
        both = []
        for f in (call, graph.replay):
            d["S"].copy_(S0)
            y.fill_(7.0)
            f()
            torch.cuda.synchronize()
            both.append((y.clone(), d["S"].clone()))
        assert torch.equal(both[0][0], both[1][0]) and torch.equal(both[0][1], both[1][1]), lens
        assert bool((both[0][0][sum(lens):] == 7).all())
        for i in range(n):
            if bounds[i] == bounds[i + 1]:
                assert torch.equal(both[0][1][i], S0[i])


@pytest.mark.parametrize("cu", [[0, 1000, 400], [0, 1400, 3], [1000, 1200, 0], [0, 1500, 1499], [600, 1, 1]])
def test_decreasing_bounds_touch_nothing_outside(cu):
    torch = torch_cuda()
    g = lib()
    say("scan decreasing bounds", cu)
    H, dk, dv, T = 16, 64, 64, 1500
    p = _problem(1, T, H, dk, dv, 1, "bf16", 2)
    d = _dev(p)
    de = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1)
    buf = torch.full((T + 128, H * dv), 3.0, dtype=torch.bfloat16, device="cuda")
    nb = g.gdnq_ssm_workspace(de, 2, T)
    ws = torch.full((nb + 256,), 0x7F, dtype=torch.uint8, device="cuda")
    g.gdnq_ssm_prefill(de, d["x"], d["B"], d["C"], d["dt"], d["A"], None, None, buf[64:64 + T], d["S"], 2, None, None,
                       torch.tensor(cu, dtype=torch.int32, device="cuda"), 2, T, ws)
    torch.cuda.synchronize()
    assert (buf[:64] == 3).all() and (buf[64 + T:] == 3).all() and (ws[nb:] == 0x7F).all()
    for i in range(2):
        if not 0 <= cu[i] < cu[i + 1] <= T:
            assert np.array_equal(d["S"][i].cpu().numpy(), p["S"][i])
