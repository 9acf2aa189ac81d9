"""The layer operators as they are used: together, from graphs, on side
streams, over pools beyond 32-bit offsets, and with memory around the
sequences that must not matter (NaN in rows of no sequence and in slots that
start anew)."""
import numpy as np
import pytest

from tests import _layer as L
from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu


class Layer:
    """A selective-state-space layer at small size: residual norm, projection
    to (z, x B C, dt), convolution over x B C, scan, gated norm.  Projections
    are torch products; every operator reads its columns in place."""

    H, dk, dv, hk, D = 4, 128, 64, 2, 192

    def __init__(self, seed):
        torch = torch_cuda()
        g = self.g = lib()
        r = np.random.default_rng(seed)
        H, dk, dv, hk, D = self.H, self.dk, self.dv, self.hk, self.D
        self.nx, self.nb = H * dv, hk * dk
        self.nc = self.nx + 2 * self.nb
        f = lambda *s, k=1.0: torch.from_numpy((r.standard_normal(s) * k).astype(np.float32)).cuda()  # noqa: E731
        self.w_in = f(D, self.nx + self.nc + H, k=D ** -0.5).bfloat16()
        self.norm_w, self.conv_w, self.conv_b, self.gate_w = f(D, k=0.1), f(4, self.nc, k=0.5), f(self.nc, k=0.1), f(self.nx, k=0.1)
        step = np.exp(r.uniform(np.log(1e-3), np.log(0.1), H))
        self.A = torch.from_numpy(-r.uniform(1, 16, H).astype(np.float32)).cuda()
        self.Dp, self.dt_bias = f(H), torch.from_numpy((step + np.log(-np.expm1(-step))).astype(np.float32)).cuda()
        self.d_norm = g.NormDesc(D=D, flags=g.NORM_RES_F32, w_offset=1.0)
        self.d_conv, self.d_ssm = g.ConvDesc(C=self.nc), g.SsmDesc(H=H, dk=dk, dv=dv, hk=hk)
        self.d_gate = g.NormDesc(D=self.nx, group=self.nx // hk, flags=g.NORM_GATE_FIRST, w_offset=1.0)

    def pool(self, n):
        torch = torch_cuda()
        return (torch.zeros(n, 3, self.nc, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(n, self.H, self.dk, self.dv, device="cuda"))

    def buffers(self, T):
        torch = torch_cuda()
        e = lambda *s, t=torch.bfloat16: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
        return dict(res=e(T, self.D, t=torch.float32), h=e(T, self.D), p=e(T, self.nx + self.nc + self.H), c=e(T, self.nc),
                    y=e(T, self.nx), o=e(T, self.nx))

    def _columns(self, b):
        z, xbc, dt = b["p"][:, :self.nx], b["p"][:, self.nx:self.nx + self.nc], b["p"][:, self.nx + self.nc:]
        c = b["c"]
        return z, xbc, dt, c[:, :self.nx], c[:, self.nx:self.nx + self.nb], c[:, self.nx + self.nb:]

    def prompts(self, b, x, res, pool, slots, cont, cu, n, T, ws):
        torch = torch_cuda()
        g = self.g
        z, xbc, dt, xs, B, C = self._columns(b)
        g.gdnq_norm_residual(self.d_norm, x, None, 1.0, res, b["res"], self.norm_w, b["h"], T)
        torch.matmul(b["h"], self.w_in, out=b["p"])
        g.gdnq_conv_prefill(self.d_conv, xbc, self.conv_w, self.conv_b, pool[0], pool[0].shape[0], slots, cont, cu, n, T,
                            b["c"])
        g.gdnq_ssm_prefill(self.d_ssm, xs, B, C, dt, self.A, self.Dp, self.dt_bias, b["y"], pool[1], pool[1].shape[0],
                           slots, cont, cu, n, T, ws)
        g.gdnq_norm_gated(self.d_gate, b["y"], z, self.gate_w, b["o"], T)

    def tokens(self, b, x, res, pool, slots, n):
        torch = torch_cuda()
        g = self.g
        z, xbc, dt, xs, B, C = self._columns(b)
        g.gdnq_norm_residual(self.d_norm, x, None, 1.0, res, b["res"], self.norm_w, b["h"], n)
        torch.matmul(b["h"], self.w_in, out=b["p"])
        g.gdnq_conv_step(self.d_conv, xbc, self.conv_w, self.conv_b, pool[0], pool[0].shape[0], slots, n, b["c"])
        g.gdnq_ssm_step(self.d_ssm, xs, B, C, dt, self.A, self.Dp, self.dt_bias, b["y"], pool[1], pool[1].shape[0], slots, n)
        g.gdnq_norm_gated(self.d_gate, b["y"], z, self.gate_w, b["o"], n)

    def workspace(self, n, T):
        torch = torch_cuda()
        return torch.empty(max(1, self.g.gdnq_ssm_workspace(self.d_ssm, n, T)), dtype=torch.uint8, device="cuda")

    def check(self, b, rows, S0, S1, conv0):
        """Every operator's output of one sequence's rows against 64 bits, from
        the buffers that it read."""
        f = lambda t: t[rows].double().cpu().numpy()  # noqa: E731
        z, xbc, dt, xs, B, C = (f(t) for t in self._columns(b))
        h64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        r = f(b["res"])
        ref = r * L.rms_rows(r, 1e-6) * (1.0 + h64(self.norm_w))
        assert not (np.abs(f(b["h"]) - ref) > np.abs(ref) * (44 * L.U + L.ROUND["bf16"])).any()
        ref, new, err = L.conv_rows(xbc, conv0, h64(self.conv_w), h64(self.conv_b), True)
        assert not (np.abs(f(b["c"]) - ref) > err + (np.abs(ref) + err) * L.ROUND["bf16"]).any()
        n, rep = len(xbc), self.H // self.hk
        heads = lambda v: np.repeat(v.reshape(n, self.hk, self.dk), rep, axis=1)  # noqa: E731
        y, S, ym, Sm, delta, v = L.ssm_rows(xs.reshape(n, self.H, self.dv), heads(B), heads(C), dt, h64(self.A),
                                            h64(self.Dp), h64(self.dt_bias), S0)
        c = np.concatenate([np.zeros((1, self.H)), np.cumsum(np.abs(delta * h64(self.A)), 0)])
        K = max((c[min(t + 64, n)] - c[t]).max() for t in range(n))
        tau = L.delta_bound(v).max() * (1 + min(K, 64)) + (self.dk + 128 + 16 * K + 16 * (n // 32 + 1)) * L.U
        bound = ym * (tau + 3 * 2.0 ** -16 + self.dk * L.U)
        got = f(b["y"]).reshape(y.shape)
        assert not (np.abs(got - y) > bound + (np.abs(y) + bound) * L.ROUND["bf16"]).any()
        assert not (np.abs(S1 - S) > Sm * (tau + 2.0 ** -24)).any()
        u = (f(b["y"]) * z * L.sigmoid(z)).reshape(n, self.hk, -1)
        ref = (u * L.rms_rows(u, 1e-6)).reshape(n, -1) * (1.0 + h64(self.gate_w))
        rel = 44 * L.U + 2 * ((2 * np.abs(z) + 8) * L.U).max()
        assert not (np.abs(f(b["o"]) - ref) > np.abs(ref) * (rel + L.ROUND["bf16"]) + 2.0 ** -120).any()
        return new


def _i32(*v):
    torch = torch_cuda()
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_prompts_then_tokens():
    """Two prompts of a packed batch, then ten tokens of each, through the
    whole layer; every operator checked against 64 bits on what it read, and
    the states handed from prompts to tokens through the pools."""
    torch = torch_cuda()
    say("layer run")
    m = Layer(1)
    lens, n_slots, extra = [70, 450], 4, 5
    T = sum(lens) + extra
    slots, cu = _i32(2, 0), _i32(0, lens[0], lens[0] + lens[1])
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, m.D, generator=gen, device="cuda").bfloat16()
    res = torch.randn(T, m.D, generator=gen, device="cuda")
    pool, b = m.pool(n_slots), m.buffers(T)
    m.prompts(b, x, res, pool, slots, None, cu, 2, T, m.workspace(2, T))
    torch.cuda.synchronize()
    S = {s: pool[1][s].double().cpu().numpy() for s in (2, 0)}
    conv = {}
    at = 0
    for s, n in zip((2, 0), lens):
        conv[s] = m.check(b, slice(at, at + n), np.zeros_like(S[s]), S[s], np.zeros((3, m.nc)))
        assert np.array_equal(conv[s], pool[0][s].double().cpu().numpy())
        at += n
    assert bool((b["c"][at:] == 7).all()) and bool((b["y"][at:] == 7).all())
    tb = m.buffers(2)
    for t in range(10):
        tx = torch.randn(2, m.D, generator=gen, device="cuda").bfloat16()
        m.tokens(tb, tx, torch.randn(2, m.D, generator=gen, device="cuda"), pool, slots, 2)
        torch.cuda.synchronize()
        for i, s in enumerate((2, 0)):
            S1 = pool[1][s].double().cpu().numpy()
            conv[s] = m.check(tb, slice(i, i + 1), S[s], S1, conv[s])
            assert np.array_equal(conv[s], pool[0][s].double().cpu().numpy())
            S[s] = S1
    assert not pool[1][1].any() and not pool[1][3].any()


def test_scan_state_through_the_codec():
    """The scan's states are states of gdnq.h: stored in 8 bits and restored,
    each value is within half a step c_j s_i of itself, and tokens go on."""
    torch = torch_cuda()
    g = lib()
    say("layer codec")
    H, dk, dv, T = 3, 128, 64, 100
    r = np.random.default_rng(8)
    t = lambda *s, k=1.0: torch.from_numpy((r.standard_normal(s) * k).astype(np.float32)).cuda().bfloat16()  # noqa: E731
    x, B, C, dt = t(T, H * dv), t(T, dk, k=0.5), t(T, dk, k=0.5), t(T, H, k=0.5)
    A, S, y = -torch.ones(H, device="cuda"), torch.zeros(1, H, dk, dv, device="cuda"), torch.empty_like(x)
    d = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1)
    g.gdnq_ssm_prefill(d, x, B, C, dt, A, None, None, y, S, 1, None, None, _i32(0, T), 1, T)
    qd = g.Desc(B=1, H=H, dk=dk, dv=dv)
    st = g.alloc_state(qd)
    back = torch.empty_like(S)
    g.gdn_state_quantize(qd, S, st)
    g.gdn_state_dequantize(qd, st, back)
    torch.cuda.synchronize()
    step = st["row_scale"].view(H, dk, 1).double() * st["col_scale"].view(H, 1, dv).double()
    assert bool(((back[0] - S[0]).abs().double() <= 0.5 * step * (1 + 1e-5)).all())
    g.gdnq_ssm_step(d, x[:1], B[:1], C[:1], dt[:1], A, None, None, y[:1], back, 1, None, 1)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y[:1].float()).all()) and bool(torch.isfinite(back).all())


def test_convolution_in_front_of_the_delta_rule():
    """Convolution, gdn_prefill, gated norm per head with a shared weight: the
    Gated DeltaNet layer's chain, its outer two against 64 bits on what they
    read, and the norm in place of a strided gate."""
    torch = torch_cuda()
    g = lib()
    say("layer delta rule")
    Bn, T, H, hk, D = 1, 96, 4, 2, 64
    nq = hk * D
    r = np.random.default_rng(4)
    t = lambda *s, k=1.0: torch.from_numpy((r.standard_normal(s) * k).astype(np.float32)).cuda()  # noqa: E731
    C = 2 * nq + H * D
    p = t(T, C + H * D).bfloat16()
    qkv, z = p[:, :C], p[:, C:]
    w, y = t(4, C, k=0.5), torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(1, 3, C, dtype=torch.bfloat16, device="cuda")
    g.gdnq_conv_prefill(g.ConvDesc(C=C), qkv, w, None, state, 1, None, None, _i32(0, T), 1, T, y)
    norm = lambda v: torch.nn.functional.normalize(v.float(), dim=-1).bfloat16().contiguous()  # noqa: E731
    q, k = norm(y[:, :nq].reshape(Bn, T, hk, D)), norm(y[:, nq:2 * nq].reshape(Bn, T, hk, D))
    v = y[:, 2 * nq:].reshape(Bn, T, H, D).contiguous()
    S, o = torch.zeros(Bn, H, D, D, device="cuda"), torch.empty(Bn, T, H, D, dtype=torch.bfloat16, device="cuda")
    a, b = torch.full((Bn, T, H), 0.95, device="cuda"), torch.full((Bn, T, H), 0.5, device="cuda")
    g.gdn_prefill(g.Desc(B=Bn, H=H, dk=D, dv=D, io_dtype=g.IO_BF16, hk=hk), S, q, k, v, a, b, o, T)
    wn, out = t(D, k=0.1) + 1.0, torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda")
    d = g.NormDesc(D=H * D, group=D, flags=g.NORM_GROUP_WEIGHT, eps=1e-6)
    g.gdnq_norm_gated(d, o.view(T, H, D), z, wn, out, T)
    torch.cuda.synchronize()
    h = lambda x: x.double().cpu().numpy()  # noqa: E731
    ref, _, err = L.conv_rows(h(qkv), np.zeros((3, C)), h(w), None, True)
    assert not (np.abs(h(y) - ref) > err + (np.abs(ref) + err) * L.ROUND["bf16"]).any()
    o64, z64 = h(o).reshape(T, H, D), h(z).reshape(T, H, D)
    assert np.abs(o64).max() > 0
    ref = o64 * L.rms_rows(o64, 1e-6) * h(wn) * z64 * L.sigmoid(z64)
    rel = 44 * L.U + (2 * np.abs(z64) + 8) * L.U
    assert not (np.abs(h(out).reshape(ref.shape) - ref) > np.abs(ref) * (rel + L.ROUND["bf16"]) + 2.0 ** -120).any()


@pytest.mark.parametrize("what", ["prompts", "tokens"])
def test_graph_replay_matches_eager(what):
    """The operators captured into a graph and replayed three times, with
    fresh inputs, eager twins and synchronizations between the replays: every
    kernel is deterministic, so outputs and pools are equal bit for bit.  The
    prompts' workspace is shared with a second graph and an eager call."""
    torch = torch_cuda()
    say("layer graph", what)
    m = Layer(2)
    T, n = (700, 2) if what == "prompts" else (3, 3)
    cu, slots = _i32(0, 130, 690), _i32(1, 0, 2)
    cont = _i32(1, 0)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, res = torch.empty(T, m.D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, m.D, device="cuda")
    pools, bufs, ws = [m.pool(3) for _ in range(3)], [m.buffers(T) for _ in range(3)], m.workspace(2, T)
    g = m.g

    def fill():
        x.copy_(torch.randn(T, m.D, generator=gen, device="cuda"))
        res.copy_(torch.randn(T, m.D, generator=gen, device="cuda"))

    def project(i):   # the library product stays outside the graph
        g.gdnq_norm_residual(m.d_norm, x, None, 1.0, res, bufs[i]["res"], m.norm_w, bufs[i]["h"], T)
        torch.matmul(bufs[i]["h"], m.w_in, out=bufs[i]["p"])

    def own(i):
        b, pool = bufs[i], pools[i]
        z, xbc, dt, xs, B, C = m._columns(b)
        if what == "prompts":
            g.gdnq_conv_prefill(m.d_conv, xbc, m.conv_w, m.conv_b, pool[0], 3, slots, cont, cu, 2, T, b["c"])
            g.gdnq_ssm_prefill(m.d_ssm, xs, B, C, dt, m.A, m.Dp, m.dt_bias, b["y"], pool[1], 3, slots, cont, cu, 2, T, ws)
        else:
            g.gdnq_conv_step(m.d_conv, xbc, m.conv_w, m.conv_b, pool[0], 3, slots, n, b["c"])
            g.gdnq_ssm_step(m.d_ssm, xs, B, C, dt, m.A, m.Dp, m.dt_bias, b["y"], pool[1], 3, slots, n)
        g.gdnq_norm_gated(m.d_gate, b["y"], z, m.gate_w, b["o"], T)

    fill()
    for i in range(3):
        project(i)
        own(i)
    torch.cuda.synchronize()
    graphs = []
    for i in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            own(i)
    torch.cuda.synchronize()
    for rep in range(3):
        say("replay", what, rep)
        fill()
        for i in range(3):
            project(i)
        torch.cuda.synchronize()
        graphs[0].replay()
        own(2)
        graphs[1].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            for k in ("c", "y", "o"):
                assert torch.equal(bufs[i][k], bufs[2][k]), (rep, i, k)
            assert torch.equal(pools[i][0], pools[2][0]) and torch.equal(pools[i][1], pools[2][1]), (rep, i)


def test_two_streams_at_once():
    """Two layers' prompts on two streams, each with its own buffers and
    workspace, give what they give one after the other."""
    torch = torch_cuda()
    say("layer streams")
    m = Layer(6)
    T, cu = 900, _i32(0, 520, 900)
    gen = torch.Generator(device="cuda").manual_seed(9)
    ins = [(torch.randn(T, m.D, generator=gen, device="cuda").bfloat16(), torch.randn(T, m.D, generator=gen, device="cuda"))
           for _ in range(2)]
    want = []
    for x, res in ins:
        pool, b = m.pool(2), m.buffers(T)
        m.prompts(b, x, res, pool, None, None, cu, 2, T, m.workspace(2, T))
        want.append((b, pool))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [(m.buffers(T), m.pool(2), m.workspace(2, T)) for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(3):
        for s, (x, res), (b, pool, ws) in zip(streams, ins, got):
            with torch.cuda.stream(s):
                m.prompts(b, x, res, pool, None, None, cu, 2, T, ws)
    torch.cuda.synchronize()
    for (wb, wp), (b, pool, _) in zip(want, got):
        for k in ("c", "y", "o"):
            assert torch.equal(b[k], wb[k]), k
        assert torch.equal(pool[0], wp[0]) and torch.equal(pool[1], wp[1])


def test_what_lies_around_the_sequences_does_not_matter():
    """NaN and infinities in rows of no sequence, in slots that start anew and
    in the workspace change nothing."""
    torch = torch_cuda()
    g = lib()
    say("layer poison")
    H, dk, dv, hk, T, C, n_slots = 4, 128, 64, 1, 800, 128, 3
    cu, slots, cont = _i32(7, 60, 60, 777), _i32(2, 1, 0), _i32(0, 1, 0)
    r = np.random.default_rng(2)
    t = lambda *s, k=1.0: torch.from_numpy((r.standard_normal(s) * k).astype(np.float32)).cuda()  # noqa: E731
    rows = {k: t(T, w, k=0.5).bfloat16() for k, w in (("x", H * dv), ("B", dk), ("C", dk), ("dt", H), ("u", C))}
    A, S, state, w = -1.0 - t(H).abs(), t(n_slots, H, dk, dv), t(n_slots, 3, C).bfloat16(), t(4, C)
    ds, dc = g.SsmDesc(H=H, dk=dk, dv=dv, hk=hk), g.ConvDesc(C=C)
    outs = []
    for poison in (None, float("nan"), float("inf")):
        q = {k: v.clone() for k, v in rows.items()}
        S1, st1 = S.clone(), state.clone()
        ws = torch.zeros(g.gdnq_ssm_workspace(ds, 3, T), dtype=torch.uint8, device="cuda")
        assert ws.numel() > 0
        if poison is not None:
            for v in q.values():
                v[:7] = poison
                v[777:] = poison
            S1[2], S1[0], st1[2], st1[0] = poison, poison, poison, poison
            ws.view(torch.float32).fill_(poison)
        y, c = torch.zeros(T, H * dv, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
        g.gdnq_ssm_prefill(ds, q["x"], q["B"], q["C"], q["dt"], A, None, None, y, S1, n_slots, slots, cont, cu, 3, T, ws)
        g.gdnq_conv_prefill(dc, q["u"], w, None, st1, n_slots, slots, cont, cu, 3, T, c)
        torch.cuda.synchronize()
        outs.append((y, S1, c, st1))
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)
    assert bool(torch.isfinite(outs[0][1]).all())


def test_offsets_beyond_32_bits():
    """Slots whose states lie behind 2^31 values, and rows 2^31 values behind
    the first, give what they give near the start."""
    torch = torch_cuda()
    g = lib()
    say("layer far offsets")
    H, dk, dv, T = 8, 128, 64, 600
    far = 2 ** 31 // (H * dk * dv) + 2
    r = np.random.default_rng(1)
    t = lambda *s, k=1.0: torch.from_numpy((r.standard_normal(s) * k).astype(np.float32)).cuda()  # noqa: E731
    ld = 1 << 22
    wide = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    x, B, C, dt = t(T, H * dv).bfloat16(), t(T, dk, k=0.5).bfloat16(), t(T, dk, k=0.5).bfloat16(), t(T, H).bfloat16()
    cols, at = {}, 0
    for k, v in (("x", x), ("B", B), ("C", C), ("dt", dt)):
        cols[k] = wide[:, at:at + v.shape[1]]
        cols[k].copy_(v)
        at += v.shape[1]
    A, S0 = -1.0 - t(H).abs(), t(H, dk, dv)
    S = torch.empty(far + 1, H, dk, dv, device="cuda")
    S[far] = S0
    d = g.SsmDesc(H=H, dk=dk, dv=dv, hk=1)
    res = []
    for q, pool, slot in (({"x": x, "B": B, "C": C, "dt": dt}, S0[None].clone(), 0), (cols, S, far)):
        y = torch.empty(T, H * dv, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(g.gdnq_ssm_workspace(d, 1, T), dtype=torch.uint8, device="cuda")
        g.gdnq_ssm_prefill(d, q["x"], q["B"], q["C"], q["dt"], A, None, None, y, pool, pool.shape[0], _i32(slot), _i32(1),
                           _i32(0, T), 1, T, ws)
        y1 = torch.empty(1, H * dv, dtype=torch.bfloat16, device="cuda")
        g.gdnq_ssm_step(d, q["x"][-1:], q["B"][-1:], q["C"][-1:], q["dt"][-1:], A, None, None, y1, pool, pool.shape[0],
                        _i32(slot), 1)
        n = torch.empty_like(x)
        g.gdnq_norm_gated(g.NormDesc(D=H * dv), q["x"], None, torch.ones(H * dv, device="cuda"), n, T)
        st = torch.zeros(1, 3, H * dv, dtype=torch.bfloat16, device="cuda")
        c = torch.empty_like(x)
        g.gdnq_conv_prefill(g.ConvDesc(C=H * dv), q["x"], torch.ones(4, H * dv, device="cuda"), None, st, 1, None, None,
                            _i32(0, T), 1, T, c)
        torch.cuda.synchronize()
        res.append((y, y1, pool[slot].clone(), n, c, st))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_binding_on_a_side_stream_argument():
    """stream= takes a torch stream; work is ordered behind what the stream holds."""
    torch = torch_cuda()
    g = lib()
    say("layer stream argument")
    x = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(10):
            x = x * 1.0001
        xb = x.bfloat16()
    y = torch.empty_like(xb)
    y.record_stream(s)
    s.wait_stream(torch.cuda.current_stream())
    w = torch.ones(4096, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    g.gdnq_norm_gated(g.NormDesc(D=4096), xb, None, w, y, 4096, stream=s)
    torch.cuda.synchronize()
    ref = xb.double() * torch.rsqrt(xb.double().square().mean(1, keepdim=True) + 1e-6)
    assert bool(((y.double() - ref).abs() <= ref.abs() * (44 * L.U + L.ROUND["bf16"])).all())
