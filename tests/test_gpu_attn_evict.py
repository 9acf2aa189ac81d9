"""Eviction from the paged cache (gdnq_kv_evict) against its definition: which
rows leave and where the others go, bit for bit; everything else stays."""
import numpy as np
import pytest

from tests import _attn as L
from tests._attn_gpu import Cache, io_of, same, up
from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu


def call(C, budget, sink, recent, H=None):
    torch = torch_cuda()
    g = lib()
    n = len(C.slots)
    desc = g.AttnDesc(H=H or C.hk, hk=C.hk, d=C.d, io_dtype=io_of(C.io), page=C.page)
    nb = g.gdnq_kv_evict_workspace(desc, C.kv(), budget, n)
    ws = torch.full((nb // 4 + 64,), -1, dtype=torch.int32, device="cuda")
    g.gdnq_kv_evict(desc, C.kv(), budget, sink, recent, C.slotsd, n, ws[:nb // 4] if nb else None)
    torch.cuda.synchronize()
    assert (ws[nb // 4:] == -1).all()


def check(C, budget, sink, recent, skip=()):
    want = [t.clone() for t in (C.k, C.v, C.acc, C.pos)]
    for i, n in enumerate(C.lens_list):
        if n <= budget or i in skip:
            continue
        pg, off = C.where(i)
        for h in range(C.hk):
            holes, kept = L.evict(C.acc[pg, h, off].numpy(), C.pos[pg, h, off].numpy(), budget, sink, recent)
            assert len(holes) == len(kept)
            for t in want:
                t[pg[holes], h, off[holes]] = t[pg[kept], h, off[kept]]
    for a, b, name in zip((C.kd, C.vd, C.accd, C.posd), want, ("k", "v", "acc", "pos")):
        assert same(a, b), name


CASES = [
    # io, hk, d, page, lens, budget, sink, recent, layout
    ("bf16", 1, 64, 8, [2], 1, 0, 0, "hr"),
    ("bf16", 2, 128, 16, [65, 64, 63, 1, 0, 66], 64, 4, 16, "hr"),
    ("f32", 3, 64, 8, [300, 41, 40, 39], 40, 2, 8, "pad"),
    ("bf16", 4, 256, 32, [500, 1000, 100], 100, 16, 40, "rh"),
    ("bf16", 8, 128, 64, [2049] * 5 + [2048, 7], 2048, 4, 128, "hr"),
    ("bf16", 1, 128, 128, [9000, 4000], 3000, 4, 200, "hr"),
    ("f32", 1, 64, 16, [1000, 70], 60, 60, 0, "hr"),
    ("bf16", 2, 64, 16, [1000, 70], 60, 0, 60, "hr"),
    ("bf16", 1, 64, 16, [70000], 30000, 1, 1, "hr"),
    ("bf16", 2, 64, 8, [20] * 200, 13, 1, 3, "hr"),
    ("bf16", 1, 64, 8, [33000], 32900, 0, 0, "hr"),
    ("bf16", 1, 64, 8, [33000], 32999, 3, 50, "hr"),
    ("bf16", 2, 64, 16, [40003, 36000, 35001], 35000, 4, 50, "rh"),
    ("f32", 3, 64, 64, [65536, 100], 90, 0, 7, "hr"),
    ("bf16", 1, 64, 32, [20000, 17001], 9000, 4, 100, "hr"),
    ("bf16", 1, 64, 16, [30001, 32768, 5], 2000, 0, 64, "hr"),
]


IDS = [f"{c[0]}-hk{c[1]}-d{c[2]}-p{c[3]}-n{len(c[4])}x{max(c[4])}-b{c[5]}-{c[8]}" for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("sums", ["random", "few values", "equal", "signs"])
def test_evict(case, sums):
    torch = torch_cuda()
    io, hk, d, page, lens, budget, sink, recent, layout = case
    say("evict", case, sums)
    rng = np.random.default_rng(page + len(lens) + budget)
    # positions in no order, gaps among them
    C = Cache(rng, lens, hk, d, page, io, layout, positions=lambda i, m: rng.permutation(2 * m + 5)[:m])
    held = ~torch.isnan(C.acc)
    if sums == "few values":
        C.acc = torch.where(held, (C.acc * 4).floor() / 4, C.acc)
    elif sums == "equal":
        C.acc = torch.where(held, torch.full_like(C.acc, 0.5), C.acc)
    elif sums == "signs":
        C.acc = torch.where(held, (C.acc * 6).floor() - 3.0, C.acc)
        half = torch.from_numpy(rng.random(tuple(C.acc.shape)) < 0.5)
        C.acc = torch.where(held & (C.acc == 0.0) & half, -C.acc, C.acc)
        C.acc = torch.where(held & (C.acc == 2.0), torch.full_like(C.acc, float("inf")), C.acc)
    C.accd = C.acc.cuda()
    call(C, budget, sink, recent)
    check(C, budget, sink, recent)


def test_more_protected_than_kept():
    """Positions that repeat: more rows are protected than the budget holds; the lower of them leave."""
    say("evict protected")
    rng = np.random.default_rng(2)
    C = Cache(rng, [90, 90], 2, 64, 16, "bf16", positions=lambda i, m: np.zeros(m) if i else np.arange(m) // 30)
    call(C, 20, 1, 5)
    check(C, 20, 1, 5)


def test_positions_at_the_type_s_ends():
    say("evict far positions")
    rng = np.random.default_rng(4)

    def far(i, m):
        return rng.permutation(np.concatenate([np.arange(m // 2) - 2 ** 31, 2 ** 31 - 1 - np.arange(m - m // 2)]))

    C = Cache(rng, [101, 50], 2, 64, 16, "bf16", positions=far)
    call(C, 40, 10, 7)
    check(C, 40, 10, 7)
    D = Cache(rng, [77], 1, 64, 16, "bf16", positions=lambda i, m: np.arange(m) - 2 ** 31)
    call(D, 40, 0, 33)
    check(D, 40, 0, 33)


def test_skipped_entries():
    say("evict skips")
    rng = np.random.default_rng(6)
    C = Cache(rng, [100] * 7, 2, 64, 16, "bf16", max_pages=8)
    C.slots[0], C.slots[1] = -1, C.n_slots
    C.lens[C.slots[2]], C.lens[C.slots[3]] = -100, 8 * 16 + 1
    C.table[C.slots[4], 6] = -1           # its last page
    C.table[C.slots[5], 0] = C.n_pages
    bad = C.table.copy()
    C.slotsd, C.lensd, C.tabled = up(C.slots), up(C.lens), up(bad)
    call(C, 50, 2, 9)
    check(C, 50, 2, 9, skip=(0, 1, 2, 3, 4, 5))


def test_nothing_to_evict():
    """A budget that no slot exceeds needs no workspace and moves nothing."""
    say("evict nothing")
    rng = np.random.default_rng(8)
    C = Cache(rng, [30, 32], 2, 64, 16, "bf16")
    for budget in (32, 33, 10 ** 9):
        call(C, budget, 0, 0)
        check(C, budget, 0, 0)
