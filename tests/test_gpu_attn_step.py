"""One new token's attention over the paged cache (gdnq_attn_step) against the
definition in 64 bits (tests/_attn.py): outputs within the bound of the fp32
form plus one rounding to the output type, sums of weights within that of the
weights; NaN lies wherever a row does not count."""
import numpy as np
import pytest

from tests import _attn as L
from tests._attn_gpu import Cache, f64, io_of, rand, same, strided, up
from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu


def check(C, H, q, o, got_acc, skip=(), window=0, scale=None, decay=1.0, missing=None):
    """Outputs o [n, H*d] (host) and the sums on the device against 64 bits."""
    hk, d, G = C.hk, C.d, H // C.hk
    scale = float(np.float32(d ** -0.5)) if scale is None else scale
    want_acc = None if C.acc is None else C.acc.clone()
    for i, n in enumerate(C.lens_list):
        if i in skip:
            continue
        lo = max(0, n - window) if window else 0
        pg, off = C.where(i, lo)
        there = np.ones(len(pg), bool) if missing is None else ~np.isin(np.arange(lo, n) // C.page, missing.get(i, []))
        pg, off = pg[there], off[there]
        for h in range(hk):
            qh = f64(q[i]).reshape(H, d)[h * G:(h + 1) * G]
            ref, w, eta, err = L.attend(qh, f64(C.k[pg, h, off]), f64(C.v[pg, h, off]), scale)
            got = f64(o[i]).reshape(H, d)[h * G:(h + 1) * G]
            bad = ~(np.abs(got - ref) <= err + (np.abs(ref) + err) * L.ROUND[C.io] + 2.0 ** -120)
            assert not bad.any(), (i, h, int(bad.sum()), np.nanmax(np.abs(got - ref)), np.max(err))
            if want_acc is not None and len(pg):
                was = f64(C.acc[pg, h, off])
                s = decay * was + w.sum(0)
                got = f64(got_acc[pg, h, off])
                assert (np.abs(got - s) <= eta * w.sum(0) + (G + 3) * L.U * (was + w.sum(0))).all(), (i, h)
                want_acc[pg, h, off] = got_acc[pg, h, off]
    assert want_acc is None or same(got_acc, want_acc)


def call(C, H, q, o, window=0, scale=0.0, decay=1.0, sums=True, n=None):
    torch = torch_cuda()
    g = lib()
    n = len(C.slots) if n is None else n
    desc = g.AttnDesc(H=H, hk=C.hk, d=C.d, io_dtype=io_of(C.io), page=C.page, window=window, scale=scale,
                      acc_decay=decay)
    kv = C.kv() if sums else C.kv(acc=None)
    nb = g.gdnq_attn_workspace(desc, kv, n)
    # the workspace is whatever it was: NaN in every word, and room around it that stays
    ws = torch.full((nb // 4 + 64,), float("nan"), device="cuda")
    g.gdnq_attn_step(desc, kv, q, o, C.slotsd, n, ws[:nb // 4] if nb else None)
    torch.cuda.synchronize()
    assert torch.isnan(ws[nb // 4:]).all()


CASES = [
    # io, H, hk, d, page, lens, window, layout, offset of the rows
    ("bf16", 1, 1, 64, 8, [1], 0, "hr", 0),
    ("bf16", 4, 1, 128, 16, [0, 1, 2, 15, 16, 17, 31, 32, 33, 0], 0, "hr", 0),
    ("bf16", 16, 2, 256, 16, [700, 3], 0, "hr", 0),
    ("bf16", 32, 8, 128, 64, [65, 127, 128, 129, 1000, 511], 0, "rh", 8),
    ("bf16", 5, 1, 64, 32, [100, 1, 300], 0, "pad", 3),
    ("bf16", 48, 2, 128, 8, [77, 260], 0, "hr", 0),          # 24 heads to a cache head
    ("bf16", 17, 1, 64, 16, [40, 513], 0, "hr", 0),
    ("bf16", 130, 2, 64, 16, [1, 97], 0, "hr", 0),
    ("f32", 6, 3, 64, 8, [5, 64, 200, 1], 0, "pad", 0),
    ("f32", 8, 8, 128, 32, [33, 150], 0, "hr", 0),
    ("f32", 20, 1, 256, 16, [129, 31], 0, "rh", 4),
    ("bf16", 8, 2, 128, 16, [1, 16, 17, 50, 300], 17, "hr", 0),
    ("f32", 8, 4, 64, 64, [1000, 63, 64, 65], 1, "hr", 0),
    ("bf16", 2, 1, 128, 128, [129, 999], 128, "hr", 0),
    ("bf16", 8, 8, 128, 65536, [70000, 3], 0, "hr", 0),
    ("bf16", 8, 1, 128, 16, [4097, 9000, 20], 0, "hr", 0),
    ("f32", 4, 2, 64, 16, [5000], 0, "hr", 0),
    ("bf16", 4, 2, 64, 8, [9] * 300 + [2000, 1], 0, "hr", 0),
    # many query heads to a cache head
    ("bf16", 64, 1, 128, 64, [3000, 1, 0, 777, 130], 0, "hr", 0),
    ("bf16", 40, 1, 64, 8, [2000, 33], 500, "rh", 3),
    # many short caches
    ("bf16", 16, 8, 128, 16, [(37 * i) % 513 for i in range(130)], 0, "hr", 0),
    ("bf16", 6, 2, 64, 8, [(11 * i) % 300 for i in range(515)], 0, "rh", 1),
    ("f32", 5, 1, 64, 16, [(5 * i) % 257 for i in range(1030)], 33, "hr", 4),
    ("bf16", 40, 2, 256, 32, [(91 * i) % 480 for i in range(260)], 0, "hr", 8),
    ("f32", 24, 8, 128, 64, [(29 * i) % 250 for i in range(128)], 0, "pad", 0),
]
IDS = [f"{c[0]}-{c[1]}x{c[2]}-d{c[3]}-p{c[4]}-n{len(c[5])}x{max(c[5])}-w{c[6]}-{c[7]}" for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("sums", [False, True])
def test_step(case, sums):
    torch = torch_cuda()
    io, H, hk, d, page, lens, window, layout, off = case
    say("attention", case, sums)
    rng = np.random.default_rng(d + page + len(lens) + H)
    C = Cache(rng, lens, hk, d, page, io, layout, sums=sums)
    q = rand(rng, (len(lens), H * d), io, 2.0)
    qd, _ = strided(q, off, 8)
    od, obuf = strided(torch.full_like(q, 0.25), off, 8)
    before = obuf.clone()
    call(C, H, qd, od, window=window, sums=sums)
    check(C, H, q, od.cpu(), None if not sums else C.accd.cpu(), window=window)
    assert same(C.kd, C.k) and same(C.vd, C.v) and (not sums or same(C.posd, C.pos))
    obuf[:, off:off + H * d] = before[:, off:off + H * d]
    assert torch.equal(obuf, before)


WIDE = [
    # io, H, hk, d, page, lens, window, layout, offset of the rows: caches that may hold 131072 rows
    ("bf16", 64, 1, 128, 64, [3000, 1, 0, 777, 130], 0, "hr", 0),
    ("bf16", 40, 1, 64, 8, [2000, 33, 5, 0], 500, "rh", 3),
    ("bf16", 32, 1, 128, 16, [1, 128, 129, 5000], 0, "hr", 0),
    ("f32", 66, 2, 64, 16, [700, 64, 65], 0, "hr", 0),
    ("bf16", 130, 2, 64, 32, [400, 90, 2500], 100, "hr", 0),
    ("bf16", 100, 1, 256, 32, [600, 5, 2000, 1], 0, "pad", 8),
    ("f32", 32, 1, 256, 16, [300, 1000, 2, 64], 0, "hr", 0),
    ("f32", 17, 1, 128, 64, [300, 1000, 2, 64], 70, "rh", 0),
]


@pytest.mark.parametrize("case", WIDE, ids=[f"{c[0]}-{c[1]}x{c[2]}-d{c[3]}-p{c[4]}-n{len(c[5])}-w{c[6]}" for c in WIDE])
@pytest.mark.parametrize("sums", [False, True])
def test_many_query_heads(case, sums):
    """More than 16 query heads to a cache head in tables wide enough for several
    groups of 16 to share a workgroup."""
    torch = torch_cuda()
    io, H, hk, d, page, lens, window, layout, off = case
    say("attention, many query heads", case, sums)
    rng = np.random.default_rng(d + page + len(lens) + H)
    C = Cache(rng, lens, hk, d, page, io, layout, sums=sums, max_pages=131072 // page)
    q = rand(rng, (len(lens), H * d), io, 2.0)
    qd, _ = strided(q, off, 8)
    od, obuf = strided(torch.full_like(q, 0.25), off, 8)
    before = obuf.clone()
    call(C, H, qd, od, window=window, sums=sums)
    check(C, H, q, od.cpu(), None if not sums else C.accd.cpu(), window=window)
    obuf[:, off:off + H * d] = before[:, off:off + H * d]
    assert torch.equal(obuf, before)


def test_skipped_entries():
    """Slots and lengths outside their range: nothing is written; pages outside the pool: their rows do not count,
    and an entry of no other rows gives zeros."""
    torch = torch_cuda()
    say("attention skips")
    rng = np.random.default_rng(1)
    C = Cache(rng, [40, 50, 60, 70, 100, 20, 33], 2, 128, 16, "bf16", max_pages=8)
    C.slots[0], C.slots[1] = -1, C.n_slots
    C.lens[C.slots[2]], C.lens[C.slots[3]] = -1, 8 * 16 + 1
    C.table[C.slots[4], 2], C.table[C.slots[4], 6] = -5, C.n_pages
    C.table[C.slots[5], :2] = 2 ** 31 - 1
    C.table[C.slots[6], 2] = -1   # the last page, one row of it
    C.slotsd, C.lensd, C.tabled = up(C.slots), up(C.lens), up(C.table)
    q = rand(rng, (7, 4 * 128), "bf16")
    o = torch.full((7, 4 * 128), 9.0, dtype=torch.bfloat16, device="cuda")
    call(C, 4, q.cuda(), o)
    assert (o[:4] == 9.0).all() and (o[5] == 0.0).all()
    check(C, 4, q, o.cpu(), C.accd.cpu(), skip=(0, 1, 2, 3), missing={4: [2, 6], 5: [0, 1], 6: [2]})


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("scale,decay,big", [(0.3, 0.5, 1.0), (1e-3, 0.0, 1.0), (0.088388, 1.0, 30.0)])
def test_scales(io, scale, decay, big):
    """Own scales and decays of the sums; scores in the thousands, where one row takes all the weight."""
    torch = torch_cuda()
    say("attention scales", io, scale, decay, big)
    rng = np.random.default_rng(7)
    C = Cache(rng, [300, 64, 1], 2, 128, 32, io)
    q = rand(rng, (3, 6 * 128), io, big)
    o = torch.zeros(3, 6 * 128, dtype=q.dtype, device="cuda")
    call(C, 6, q.cuda(), o, scale=scale, decay=decay)
    check(C, 6, q, o.cpu(), C.accd.cpu(), scale=float(np.float32(scale)), decay=decay)


@pytest.mark.parametrize("lens", [[300, 64, 1, 0], [70, 128, 3, 9]])
def test_sums_replaced(lens):
    """A decay of 0 replaces the sums without reading them."""
    torch = torch_cuda()
    say("attention sums replaced", lens)
    rng = np.random.default_rng(8)
    C = Cache(rng, lens, 2, 64, 16, "bf16")
    q = rand(rng, (4, 6 * 64), "bf16", 2.0)
    o = torch.zeros(4, 6 * 64, dtype=q.dtype, device="cuda")
    C.acc.fill_(0.0)
    C.accd.fill_(float("nan"))
    call(C, 6, q.cuda(), o, decay=0.0)
    got = C.accd.cpu()
    for i in range(4):
        pg, off = C.where(i)
        assert not torch.isnan(got[pg, :, off]).any()
    check(C, 6, q, o.cpu(), torch.where(torch.isnan(got), torch.zeros_like(got), got), decay=0.0)


def test_one_slot_twice():
    """Entries of one slot (two tokens that attend to the same rows)."""
    torch = torch_cuda()
    say("attention, one slot twice")
    rng = np.random.default_rng(14)
    C = Cache(rng, [500, 40], 2, 64, 16, "bf16", sums=False)
    C.slots, C.lens_list = C.slots[[0, 1, 0, 0]], [500, 40, 500, 500]
    C.slotsd = up(C.slots)
    q = rand(rng, (4, 8 * 64), "bf16", 2.0)
    o = torch.zeros(4, 8 * 64, dtype=q.dtype, device="cuda")
    call(C, 8, q.cuda(), o, sums=False)
    check(C, 8, q, o.cpu(), None)


def test_equal_and_low_scores():
    """Equal rows share the weight; scores near the type's lowest value, and among them one high one."""
    torch = torch_cuda()
    say("attention low scores")
    rng = np.random.default_rng(9)
    C = Cache(rng, [200, 200, 200], 1, 64, 8, "f32")
    q = np.zeros((3, 2 * 64), np.float32)
    for i, (kk, qq) in enumerate([(0.0, 1.0), (-1e18, 1e18), (-1e18, 1e18)]):
        pg, off = C.where(i)
        C.k[pg, :, off] = 0.0
        C.k[pg, :, off, 0] = kk
        q[i, ::64] = qq
    pg, off = C.where(2)
    C.k[pg[150], 0, off[150], 0] = 0.0
    C.kd = C.k.cuda()
    o = torch.zeros(3, 128, device="cuda")
    before = C.acc.clone()
    call(C, 2, torch.from_numpy(q).cuda(), o)
    v = [C.rows(C.v, i, 0) for i in range(3)]
    got = f64(o).reshape(3, 2, 64)
    for i in (0, 1):
        assert np.abs(got[i] - v[i].mean(0)).max() <= (2 * 200 + 40) * L.U * np.abs(v[i]).mean(0).max()
        pg, off = C.where(i)
        assert np.abs(f64(C.accd.cpu()[pg, 0, off]) - f64(before[pg, 0, off]) - 2 / 200).max() < 1e-6
    assert np.array_equal(got[2], np.stack([v[2][150]] * 2))


SICK = [
    # rows of the entries, pages of a table, query heads: a wave for each pair, pieces of pairs in several shares,
    # several pairs in a share, the same with several groups of query heads in a workgroup
    ("waves", [100, 7, 128], 8, 16), ("pieces", [600, 40], 60, 16), ("whole", [600] + [590] * 520, 40, 16),
    ("groups", [600] + [590] * 120, 40, 80),
]


@pytest.mark.parametrize("what,lens,width,H", SICK, ids=[c[0] for c in SICK])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["key", "query"])
def test_nan_stays_seen(what, lens, width, H, io, where):
    """NaN in a key or a query reaches the outputs and sums of its heads, however the
    call is dealt out, and nothing else."""
    torch = torch_cuda()
    say("attention with NaN", what, io, where)
    rng = np.random.default_rng(23)
    C = Cache(rng, lens, 2, 64, 16, io, max_pages=width)
    n, G = len(lens), H // 2
    q = rand(rng, (n, H * 64), io, 2.0)
    seen = []
    for sick in (False, True):
        if sick and where == "key":
            pg, off = C.where(0)
            C.kd[int(pg[70]), 1, int(off[70]), 5] = float("nan")
        if sick and where == "query":
            q[0, (G + 3) * 64 + 9] = float("nan")
        C.accd.copy_(C.acc)
        o = torch.zeros(n, H * 64, dtype=q.dtype, device="cuda")
        call(C, H, q.cuda(), o)
        seen.append((o.reshape(n, H, 64).cpu(), C.accd.cpu()))
    (o0, a0), (o1, a1) = seen
    heads = range(G, H) if where == "key" else [G + 3]
    assert torch.isnan(o1[0, list(heads)]).all() and not torch.isnan(o0).any()
    pg, off = C.where(0)
    assert torch.isnan(a1[pg, 1, off]).all() and not torch.isnan(a0[pg, 1, off]).any()
    o1[0, list(heads)], a1[pg, 1, off] = o0[0, list(heads)], a0[pg, 1, off]
    assert same(o1, o0) and same(a1, a0)


def test_shared_pages():
    """Entries that share the pages of a common beginning."""
    torch = torch_cuda()
    say("attention shared pages")
    rng = np.random.default_rng(13)
    C = Cache(rng, [100, 100, 90], 2, 64, 16, "bf16", sums=False)
    C.table[C.slots[1], :3] = C.table[C.slots[0], :3]
    C.table[C.slots[2], :5] = C.table[C.slots[0], :5]
    C.tabled = up(C.table)
    q = rand(rng, (3, 4 * 64), "bf16")
    o = torch.zeros(3, 4 * 64, dtype=torch.bfloat16, device="cuda")
    call(C, 4, q.cuda(), o, sums=False)
    check(C, 4, q, o.cpu(), None)


@pytest.mark.parametrize("io,page", [("bf16", 8), ("bf16", 16), ("f32", 8), ("bf16", 64)])
def test_pages_before_a_window(io, page):
    """Table entries before a window are stale: pages of other entries by now, or
    none.  Nothing of them counts, and the others' sums are theirs alone."""
    torch = torch_cuda()
    say("attention, stale pages before a window", io, page)
    rng = np.random.default_rng(page)
    lens, window = [200 + 7 * i for i in range(24)], 45
    C = Cache(rng, lens, 2, 64, page, io)
    live = [set(C.table[C.slots[i], (n - window) // page:-(-n // page)].tolist()) for i, n in enumerate(lens)]
    for i, n in enumerate(lens):
        others = [p for j in range(24) if j != i for p in live[j]] + [-3, C.n_pages]
        C.table[C.slots[i], :(n - window) // page] = rng.choice(others, (n - window) // page)
    C.tabled = up(C.table)
    q = rand(rng, (24, 8 * 64), io, 2.0)
    for _ in range(3):
        C.accd.copy_(C.acc)
        o = torch.zeros(24, 8 * 64, dtype=q.dtype, device="cuda")
        call(C, 8, q.cuda(), o, window=window)
        check(C, 8, q, o.cpu(), C.accd.cpu(), window=window)


def test_repeated_calls_agree():
    """The same call gives the same bits, whatever the workspace held."""
    torch = torch_cuda()
    say("attention repeats")
    rng = np.random.default_rng(17)
    C = Cache(rng, [3000, 1, 777, 0, 64], 4, 128, 32, "bf16")
    q = rand(rng, (5, 16 * 128), "bf16").cuda()
    seen = []
    for _ in range(3):
        C.accd.copy_(C.acc)
        o = torch.zeros(5, 16 * 128, dtype=torch.bfloat16, device="cuda")
        call(C, 16, q, o)
        seen.append((o.clone(), C.accd.clone()))
    assert all(same(a, seen[0][0]) and same(b, seen[0][1]) for a, b in seen)


def test_a_marshalled_cache_says_what_it_is():
    """A cache marshalled once keeps its tensors, and is refused where the descriptor is another's."""
    torch = torch_cuda()
    g = lib()
    say("attention cache of another descriptor")
    rng = np.random.default_rng(19)
    C = Cache(rng, [20], 2, 64, 16, "bf16", extra_pages=0)
    kv = C.kv().c(g.AttnDesc(H=4, hk=2, d=64, page=16))
    q = torch.zeros(1, 8 * 64, dtype=torch.bfloat16, device="cuda")
    for other in (dict(H=4, hk=1), dict(H=8, hk=4), dict(H=4, hk=2, page=32), dict(H=4, hk=2, d=128),
                  dict(H=4, hk=2, io_dtype=g.IO_F32)):
        with pytest.raises(g.GdnqError, match="kv is a cache of"):
            g.gdnq_attn_step(g.AttnDesc(**{**dict(d=64, page=16), **other}), kv, q, q.clone(), C.slotsd, 1, None)
    with pytest.raises(g.GdnqError, match="shape and strides"):
        C.kv(v=C.vd.transpose(1, 2).contiguous().transpose(1, 2)).c(g.AttnDesc(H=4, hk=2, d=64, page=16))
    with pytest.raises(g.GdnqError, match="must be"):
        C.kv(k=C.kd[..., :32]).c(g.AttnDesc(H=4, hk=2, d=64, page=16))
    with pytest.raises(g.GdnqError, match="overlap"):
        one = C.kd[:1, :1, :1].expand(C.kd.shape)
        C.kv(k=one, v=one).c(g.AttnDesc(H=4, hk=2, d=64, page=16))
    with pytest.raises(g.GdnqError, match="acc has"):
        C.kv(acc=C.accd[:1]).c(g.AttnDesc(H=4, hk=2, d=64, page=16))
    with pytest.raises(g.GdnqError, match="lens is"):
        C.kv(lens=C.lensd.long()).c(g.AttnDesc(H=4, hk=2, d=64, page=16))


@pytest.mark.parametrize("hk,n_pages", [(1, 5), (2, 1), (1, 1)])
def test_strides_of_one(hk, n_pages):
    """A dimension of one has no distance: k and v may state other strides for it."""
    torch = torch_cuda()
    g = lib()
    say("attention cache with dimensions of one", hk, n_pages)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    k, v = (torch.randn(n_pages, hk, 16, 64, generator=gen, device="cuda").bfloat16() for _ in "kv")
    other = v.clone().as_strided(v.shape, [st if m > 1 else 8 * st + 64 for st, m in zip(v.stride(), v.shape)])
    assert other.stride() != v.stride() and torch.equal(other, v)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None].contiguous()
    lens = torch.tensor([16 * n_pages - 3], dtype=torch.int32, device="cuda")
    desc = g.AttnDesc(H=2 * hk, hk=hk, d=64, page=16)
    q = torch.randn(1, 2 * hk * 64, generator=gen, device="cuda").bfloat16()
    o = []
    for w in (v, other):
        kv = g.Kv(k, w, table, lens)
        ws = torch.empty(max(16, g.gdnq_attn_workspace(desc, kv, 1)), dtype=torch.uint8, device="cuda")
        o.append(torch.empty_like(q))
        g.gdnq_attn_step(desc, kv, q, o[-1], None, 1, ws)
    assert same(*o)
