"""The attention operators as they are used: together (prompts, then tokens
with sums of weights and eviction), from graphs, on side streams, over caches
beyond 32-bit offsets and of a million rows."""
import numpy as np
import pytest

from tests import _attn as L
from tests._attn_gpu import Cache, f64, io_of, rand, same, up
from tests._gpu import lib, say, torch_cuda
from tests.test_gpu_attn_rope import table_of
from tests.test_gpu_attn_step import check as check_step

pytestmark = pytest.mark.gpu


class Layer:
    """The attention operators of one layer at small size, over one cache: a
    prompt or a token of each entry is stored, attends, and the cache is cut
    back to its budget."""

    H, hk, d, page, width = 6, 2, 64, 8, 12
    budget, sink, recent = 40, 2, 8

    def __init__(self, n, seed, io="bf16"):
        torch = torch_cuda()
        g = self.g = lib()
        rng = np.random.default_rng(seed)
        self.n, self.io = n, io
        C = self.C = Cache(rng, [0] * n, self.hk, self.d, self.page, io, extra_pages=n * self.width + 3,
                           max_pages=self.width)
        pages = rng.permutation(C.n_pages)[:n * self.width].reshape(n, self.width)
        C.table[C.slots] = pages
        C.tabled = up(C.table)
        self.rope = g.RopeDesc(d=self.d, rot=32, io_dtype=io_of(io))
        self.freqs = table_of(self.rope)
        self.desc = g.AttnDesc(H=self.H, hk=self.hk, d=self.d, io_dtype=io_of(io), page=self.page)
        self.kv = C.kv().c(self.desc)
        ws = max(g.gdnq_attn_workspace(self.desc, self.kv, n),
                 g.gdnq_kv_evict_workspace(self.desc, self.kv, self.budget, n), 16)
        self.ws = torch.empty(ws, dtype=torch.uint8, device="cuda")
        self.slot_index = C.slotsd.long()
        self.seen = torch.zeros(n, dtype=torch.int32, device="cuda")   # tokens of each entry so far

    def token(self, qkv, o):
        """One token of each entry: columns q, k, v of qkv [n, (H + 2 hk) d]; q is turned in place."""
        g, C = self.g, self.C
        nq, nk = self.H * self.d, self.hk * self.d
        q, k, v = qkv[:, :nq], qkv[:, nq:nq + nk], qkv[:, nq + nk:]
        C.lensd.index_add_(0, self.slot_index, self.one(o))
        g.gdnq_kv_append(self.desc, self.rope, self.freqs, self.kv, q, q, k, v, self.seen, C.slotsd, None, self.n,
                         self.n)
        g.gdnq_attn_step(self.desc, self.kv, q, o, C.slotsd, self.n, self.ws)
        g.gdnq_kv_evict(self.desc, self.kv, self.budget, self.sink, self.recent, C.slotsd, self.n, self.ws)
        C.lensd.clamp_(max=self.budget)
        self.seen.add_(1)

    def one(self, o):
        if not hasattr(self, "_one"):
            self._one = torch_cuda().ones(self.n, dtype=torch_cuda().int32, device="cuda")
        return self._one

    def state(self):
        C = self.C
        return [t.clone() for t in (C.kd, C.vd, C.accd, C.posd, C.lensd, self.seen)]

    def restore(self, s):
        C = self.C
        for t, x in zip((C.kd, C.vd, C.accd, C.posd, C.lensd, self.seen), s):
            t.copy_(x)

    def pull(self):
        """The device's cache as the host's, before the next call."""
        C = self.C
        C.k, C.v, C.acc, C.pos = (t.cpu() for t in (C.kd, C.vd, C.accd, C.posd))


def test_prompts_then_tokens():
    """Every call against 64 bits, from the cache that it read."""
    torch = torch_cuda()
    say("attention layer: prompts, tokens, eviction")
    A = Layer(4, 1)
    g, C = A.g, A.C
    rng = np.random.default_rng(2)
    prompt = [30, 0, 70, 40]
    T = sum(prompt)
    cu = np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32)
    C.lens[C.slots] = prompt
    C.lensd.copy_(up(C.lens))
    C.lens_list = list(prompt)
    x = rand(rng, (T, (A.H + 2 * A.hk) * A.d), "bf16").cuda()
    nq, nk = A.H * A.d, A.hk * A.d
    kept = x.clone()
    g.gdnq_kv_append(A.desc, A.rope, A.freqs, A.kv, x[:, :nq], x[:, :nq], x[:, nq:nq + nk], x[:, nq + nk:], None,
                     C.slotsd, up(cu), 4, T)
    A.seen.copy_(up(np.array(prompt, np.int32)))
    A.pull()
    th = L.theta(32)
    for i, m in enumerate(prompt):
        pg, off = C.where(i)
        ref, err = L.rotate(f64(kept[cu[i]:cu[i + 1], nq:nq + nk]).reshape(m, A.hk, A.d), np.arange(m), th, 32)
        assert (np.abs(f64(C.k[pg, :, off]) - ref) <= err + (np.abs(ref) + err) * L.ROUND["bf16"]).all()
        assert torch.equal(C.v[pg, :, off], kept[cu[i]:cu[i + 1], nq + nk:].cpu().reshape(m, A.hk, A.d))
        assert (C.acc[pg, :, off] == 0).all() and (C.pos[pg, :, off] == torch.arange(m)[:, None]).all()
    for step in range(14):
        x = rand(rng, (4, (A.H + 2 * A.hk) * A.d), "bf16", 1.5).cuda()
        o = torch.empty(4, nq, dtype=torch.bfloat16, device="cuda")
        C.lens_list = [m + 1 for m in C.lens_list]
        C.lensd.index_add_(0, A.slot_index, A.one(o))
        before = x.clone()
        seen = A.seen.cpu().numpy()
        g.gdnq_kv_append(A.desc, A.rope, A.freqs, A.kv, x[:, :nq], x[:, :nq], x[:, nq:nq + nk], x[:, nq + nk:], A.seen,
                         C.slotsd, None, 4, 4)
        ref, err = L.rotate(f64(before[:, :nq]).reshape(4, A.H, A.d), seen, th, 32)
        assert (np.abs(f64(x[:, :nq]).reshape(ref.shape) - ref) <= err + (np.abs(ref) + err) * L.ROUND["bf16"]).all()
        A.pull()
        g.gdnq_attn_step(A.desc, A.kv, x[:, :nq], o, C.slotsd, 4, A.ws)
        check_step(C, A.H, x[:, :nq].cpu(), o.cpu(), C.accd.cpu())
        A.pull()
        g.gdnq_kv_evict(A.desc, A.kv, A.budget, A.sink, A.recent, C.slotsd, 4, A.ws)
        want = [t.clone() for t in (C.k, C.v, C.acc, C.pos)]
        for i, m in enumerate(C.lens_list):
            if m <= A.budget:
                continue
            pg, off = C.where(i)
            for h in range(A.hk):
                holes, moved = L.evict(C.acc[pg, h, off].numpy(), C.pos[pg, h, off].numpy(), A.budget, A.sink, A.recent)
                for t in want:
                    t[pg[holes], h, off[holes]] = t[pg[moved], h, off[moved]]
        assert all(same(a, b) for a, b in zip((C.kd, C.vd, C.accd, C.posd), want))
        C.lens_list = [min(m, A.budget) for m in C.lens_list]
        C.lensd.clamp_(max=A.budget)
        A.seen.add_(1)
        # the sinks and the newest tokens are still there
        A.pull()
        for i, m in enumerate(C.lens_list):
            pg, off = C.where(i)
            for h in range(A.hk):
                p = set(C.pos[pg, h, off].tolist())
                s = int(A.seen[i])
                assert len(p) == m and set(range(max(0, s - A.recent), s)) <= p and set(range(min(A.sink, s))) <= p


# a pool of both caches: its shape, made from pages n, heads h, rows r, values d and "2", with keys and values there
ORDERS = ["n2hrd", "nh2rd", "nhr2d", "nr2hd", "nrh2d", "n2rhd"]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_one_pool_of_keys_and_values(order, io):
    """Keys and values between each other's pages, heads or rows give what two pools give, bit for bit."""
    torch = torch_cuda()
    say("attention, one pool", order, io)
    A, B = Layer(5, 31, io), Layer(5, 31, io)
    C = B.C
    size = dict(zip("n2hrd", (C.n_pages, 2, B.hk, B.page, B.d)))
    pool = torch.full([size[x] for x in order], float("nan"), dtype=C.kd.dtype, device="cuda")
    k, v = (pool.select(order.index("2"), i).permute([order.replace("2", "").index(x) for x in "nhrd"]) for i in (0, 1))
    k.copy_(C.kd)
    v.copy_(C.vd)
    C.kd, C.vd = k, v
    B.kv = C.kv().c(B.desc)
    rng = np.random.default_rng(32)
    width = (A.H + 2 * A.hk) * A.d
    prompt = [30, 0, 70, 96, 1]
    cu = up(np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32))
    x = rand(rng, (sum(prompt), width), io).cuda()
    tokens = [rand(rng, (5, width), io).cuda() for _ in range(20)]
    seen = []
    for M in (A, B):
        M.C.lensd[M.slot_index] = up(np.array(prompt, np.int32))
        nq, nk = M.H * M.d, M.hk * M.d
        y = x.clone()
        M.g.gdnq_kv_append(M.desc, M.rope, M.freqs, M.kv, y[:, :nq], y[:, :nq], y[:, nq:nq + nk], y[:, nq + nk:], None,
                           M.C.slotsd, cu, 5, sum(prompt))
        M.seen.copy_(up(np.array(prompt, np.int32)))
        M.g.gdnq_kv_evict(M.desc, M.kv, M.budget, M.sink, M.recent, M.C.slotsd, 5, M.ws)
        M.C.lensd.clamp_(max=M.budget)
        o = torch.empty(5, nq, dtype=x.dtype, device="cuda")
        got = [y, *M.state()]
        for t in tokens:
            M.token(t.clone(), o)
            got += [o.clone(), *M.state()]
        seen.append(got)
    assert all(same(a, b) for a, b in zip(*seen))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_graph_replays(io):
    """A token's calls captured once and replayed, with eager work of the same
    program between the replays, give what eager calls give, bit for bit."""
    torch = torch_cuda()
    say("attention graph", io)
    A = Layer(5, 3, io)
    rng = np.random.default_rng(4)
    width = (A.H + 2 * A.hk) * A.d
    xs = [rand(rng, (5, width), io).cuda() for _ in range(12)]
    A.C.lensd.index_fill_(0, A.slot_index, 0)   # the slots in use are empty, the others stay as they are
    start = A.state()
    o = torch.empty(5, A.H * A.d, dtype=xs[0].dtype, device="cuda")
    eager = []
    for x in xs * 4:
        A.token(x.clone(), o)
        eager.append((o.clone(), A.state()))
    A.restore(start)
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        A.token(x, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.token(x, o)
    A.restore(start)
    other = Layer(5, 9, io)
    y = torch.empty_like(o)
    other.C.lensd.index_fill_(0, other.slot_index, 0)
    for i, new in enumerate(xs * 4):
        x.copy_(new)
        graph.replay()
        if i % 3 == 0:
            other.token(new.clone(), y)
            torch.cuda.synchronize()
        assert same(o, eager[i][0]), i
        assert all(same(a, b) for a, b in zip(A.state(), eager[i][1])), i


def test_two_graphs_share_a_workspace():
    """Two captured steps over two caches with one workspace, replayed in turn."""
    torch = torch_cuda()
    say("attention graphs, one workspace")
    A, B = Layer(3, 5), Layer(3, 6)
    B.ws = A.ws
    rng = np.random.default_rng(7)
    x = rand(rng, (3, (A.H + 2 * A.hk) * A.d), "bf16").cuda()
    outs, graphs, starts, bufs = [], [], [], []
    for M in (A, B):
        M.C.lensd.index_fill_(0, M.slot_index, 0)
        starts.append(M.state())
        o, buf = torch.empty(3, A.H * A.d, dtype=torch.bfloat16, device="cuda"), x.clone()
        M.token(buf, o)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            buf.copy_(x)
            M.token(buf, o)
        M.restore(starts[-1])
        outs.append(o)
        bufs.append(buf)   # the graph's, as long as it is replayed
        graphs.append(graph)
    got = []
    for _ in range(50):
        for k in (0, 1):
            graphs[k].replay()
            got.append(outs[k].clone())
    ends = [A.state(), B.state()]
    for M, s in zip((A, B), starts):
        M.restore(s)
    for i in range(50):
        for k, M in enumerate((A, B)):
            M.token(x.clone(), outs[k])
            assert same(outs[k], got[2 * i + k]), (i, k)
    assert all(same(a, b) for M, e in zip((A, B), ends) for a, b in zip(M.state(), e))


def test_two_streams():
    """Calls on two streams at once, each with its own cache and workspace."""
    torch = torch_cuda()
    say("attention on two streams")
    Ls = [Layer(40, 11), Layer(40, 12)]
    rng = np.random.default_rng(13)
    xs = [rand(rng, (40, (Ls[0].H + 2 * Ls[0].hk) * Ls[0].d), "bf16").cuda() for _ in range(3)]
    want, starts = [], []
    for M in Ls:
        M.C.lensd.index_fill_(0, M.slot_index, 0)
        starts.append(M.state())
        o = torch.empty(40, M.H * M.d, dtype=torch.bfloat16, device="cuda")
        M.one(o)
        for i in range(60):
            M.token(xs[i % 3].clone(), o)
        want.append([o.clone(), *M.state()])
        M.restore(starts[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty(40, M.H * M.d, dtype=torch.bfloat16, device="cuda") for M in Ls]
    torch.cuda.synchronize()
    for i in range(60):
        for M, s, o in zip(Ls, streams, outs):
            with torch.cuda.stream(s):
                M.token(xs[i % 3].clone(), o)
    torch.cuda.synchronize()
    for M, o, w in zip(Ls, outs, want):
        assert all(same(a, b) for a, b in zip([o, *M.state()], w))


def test_far_pages():
    """Pages beyond 2^31 elements of the pool."""
    torch = torch_cuda()
    g = lib()
    say("attention far pages")
    hk, d, page, H, n_pages = 8, 128, 64, 16, 40000
    rng = np.random.default_rng(21)
    k = torch.empty(n_pages, hk, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    acc = torch.zeros(n_pages, hk, page, device="cuda")
    pos = torch.zeros(n_pages, hk, page, dtype=torch.int32, device="cuda")
    assert k.numel() > 2 ** 31
    lens = [300, 130]
    table = np.zeros((2, 5), np.int32)
    table[0], table[1] = [39999, 35000, 33000, 2, 39998], [34000, 36001, 39000, 1, 1]
    desc = g.AttnDesc(H=H, hk=hk, d=d, page=page)
    kv = g.Kv(k, v, up(table), up(np.array(lens, np.int32)), acc, pos)
    rope = g.RopeDesc(d=d)
    T = sum(lens)
    kn, vn = rand(rng, (T, hk * d), "bf16"), rand(rng, (T, hk * d), "bf16")
    g.gdnq_kv_append(desc, rope, table_of(rope), kv, None, None, kn.cuda(), vn.cuda(), None, None,
                     up(np.array([0, 300, 430], np.int32)), 2, T)
    q = rand(rng, (2, H * d), "bf16")
    o = torch.empty(2, H * d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(g.gdnq_attn_workspace(desc, kv, 2), g.gdnq_kv_evict_workspace(desc, kv, 100, 2)),
                     dtype=torch.uint8, device="cuda")
    g.gdnq_attn_step(desc, kv, q.cuda(), o, None, 2, ws)
    th = L.theta(d)
    for i, (lo, m) in enumerate(((0, 300), (300, 130))):
        r = np.arange(m)
        pg, off = torch.from_numpy(table[i][r // page].astype(np.int64)).cuda(), torch.from_numpy(r % page).cuda()
        ref, err = L.rotate(f64(kn[lo:lo + m]).reshape(m, hk, d), r, th, d)
        kk, vv = k[pg, :, off].cpu(), v[pg, :, off].cpu()
        assert (np.abs(f64(kk) - ref) <= err + (np.abs(ref) + err) * L.ROUND["bf16"]).all()
        assert torch.equal(vv, vn[lo:lo + m].reshape(m, hk, d))
        aa = acc[pg, :, off].cpu()
        for h in range(hk):
            ref, w, eta, err = L.attend(f64(q[i]).reshape(H, d)[2 * h:2 * h + 2], f64(kk[:, h]), f64(vv[:, h]),
                                        float(np.float32(d ** -0.5)))
            got = f64(o[i]).reshape(H, d)[2 * h:2 * h + 2]
            assert (np.abs(got - ref) <= err + (np.abs(ref) + err) * L.ROUND["bf16"]).all()
            assert (np.abs(f64(aa[:, h]) - w.sum(0)) <= (eta + 5 * L.U) * w.sum(0)).all()
        g.gdnq_kv_evict(desc, kv, 100, 4, 20, None, 2, ws) if i else None
    for i, m in enumerate(lens):
        if i == 0:
            continue
        holes, moved = L.evict(aa[:, 3].numpy(), np.arange(m), 100, 4, 20)
        want = vv[:, 3].clone()
        want[holes] = want[moved]
        assert torch.equal(v[pg, 3, off].cpu(), want)


@pytest.mark.parametrize("sums", [False, True])
def test_a_million_rows(sums):
    """One entry of 1100000 rows: against 64 bits on the device.  A lane's chain of sums is a
    share's steps, and the join adds the shares: 600 + 512 + 64 additions at most."""
    torch = torch_cuda()
    g = lib()
    say("attention over a million rows", sums)
    n, d, page, H = 1100000, 64, 256, 4
    pages = -(-n // page)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    k, v = (torch.randn(pages, 1, page, d, generator=gen, device="cuda").bfloat16() for _ in "kv")
    table = torch.randperm(pages, generator=gen, device="cuda").int()[None].contiguous()
    acc = torch.zeros(pages, 1, page, device="cuda") if sums else None
    kv = g.Kv(k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"), acc)
    desc = g.AttnDesc(H=H, hk=1, d=d, page=page)
    q = (torch.randn(1, H * d, generator=gen, device="cuda") * 2).bfloat16()
    o = torch.empty_like(q)
    ws = torch.empty(g.gdnq_attn_workspace(desc, kv, 1), dtype=torch.uint8, device="cuda")
    g.gdnq_attn_step(desc, kv, q, o, None, 1, ws)
    K, V = (t[table[0].long(), 0].reshape(-1, d)[:n].double() for t in (k, v))
    s = torch.matmul(q.double().reshape(H, d), K.t().contiguous()) / 8
    w = torch.softmax(s, -1)
    ref, mag = torch.matmul(w, V), torch.matmul(w, V.abs())
    qk = float((torch.matmul(q.double().reshape(H, d).abs(), K.abs().t().contiguous()) / 8).max())
    eta = (2 * (d + 8) * qk + 8 + 2 * 1200 + 4 * float(s.max() - s.min())) * L.U + 2.0 ** -17
    err = mag * (2 * eta + 2 * 1200 * L.U)
    got = o.double().reshape(H, d)
    assert bool(((got - ref).abs() <= err + (ref.abs() + err) * L.ROUND["bf16"]).all())
    if sums:
        a, wa = acc[table[0].long(), 0].reshape(-1)[:n].double(), w.sum(0)
        assert bool(((a - wa).abs() <= (2 * eta + 1200 * L.U + 8 * L.U) * wa).all())
