"""New tokens into the paged cache (gdnq_kv_append): turned queries and keys
within the bound of tests/_attn.py, values, positions and sums exactly; every
other byte of the cache and of the queries' buffer stays as it was."""
import numpy as np
import pytest

from tests import _attn as L
from tests._attn_gpu import Cache, f64, io_of, rand, same, strided, up
from tests._gpu import lib, say, torch_cuda
from tests.test_gpu_attn_rope import table_of

pytestmark = pytest.mark.gpu

CASES = [
    # io, H, hk, d, page, rot, interleaved, layout, new tokens (None: one each), held, offset of the rows
    ("bf16", 4, 2, 64, 8, 64, False, "hr", None, [0], 0),
    ("bf16", 32, 8, 128, 16, 128, False, "hr", None, [5, 15, 16, 17, 100, 31, 0], 0),
    ("f32", 6, 3, 64, 16, 32, True, "rh", None, [3, 70, 8], 4),
    ("bf16", 16, 2, 256, 32, 64, False, "pad", None, [40, 2], 8),
    ("bf16", 5, 1, 128, 64, 100, True, "hr", None, [9, 63, 64, 127, 128], 3),
    ("bf16", 8, 2, 128, 16, 128, False, "hr", [3, 0, 1, 40, 65, 0, 16], [0, 9, 15, 7, 3, 20, 0], 0),
    ("f32", 2, 2, 64, 8, 64, True, "pad", [7, 33, 1], [1, 0, 8], 0),
    ("bf16", 24, 8, 64, 128, 0, False, "rh", [300, 1, 129], [0, 127, 5], 8),
    ("bf16", 3, 1, 256, 16, 256, False, "hr", [1] * 90 + [0, 2, 31], [5] * 93, 1),
]


IDS = [f"{c[0]}-d{c[3]}-p{c[4]}-r{c[5]}-{c[7]}-n{len(c[9])}-off{c[10]}" for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("mode", ["rows", "positions", "keys alone", "no sums"])
def test_append(case, mode):
    torch = torch_cuda()
    g = lib()
    io, H, hk, d, page, rot, inter, layout, new, held, off = case
    say("append", case, mode)
    rng = np.random.default_rng(d + page + len(held))
    packed, n = new is not None, len(held)
    new = new or [1] * n
    T = sum(new) + (4 if packed else 0)
    C = Cache(rng, [a + b for a, b in zip(held, new)], hk, d, page, io, layout, sums=mode != "no sums")
    if n > 4:
        C.slots[1], C.slots[2] = -1, C.n_slots            # skipped
        C.table[C.slots[3], (C.lens_list[3] - 1) // page] = C.n_pages   # its last page does not exist
        C.tabled, C.slotsd = up(C.table), up(C.slots)
    first = 2 if packed else 0
    cu = (np.concatenate([[0], np.cumsum(new)]) + first).astype(np.int32)
    pos = rng.integers(-100, 1 << 20, T).astype(np.int32) if mode == "positions" else None
    q, k, v = rand(rng, (T, H * d), io), rand(rng, (T, hk * d), io), rand(rng, (T, hk * d), io)
    (qd, _), (kd, _), (vd, _) = strided(q, off, 8), strided(k, off, 8), strided(v, off, 16)
    od, obuf = strided(torch.full_like(q, 0.25), off, 8)
    before = obuf.clone()
    flags = g.ROPE_INTERLEAVED if inter else 0
    rope = None if rot == 0 else g.RopeDesc(d=d, rot=rot, io_dtype=io_of(io), flags=flags)
    desc = g.AttnDesc(H=H, hk=hk, d=d, io_dtype=io_of(io), page=page)
    with_q = mode != "keys alone"
    g.gdnq_kv_append(desc, rope, None if rope is None else table_of(rope), C.kv(), qd if with_q else None,
                     od if with_q else None, kd, vd, up(pos), C.slotsd, up(cu) if packed else None, n, T)
    torch.cuda.synchronize()
    wk, wv, wacc, wpos = (None if t is None else t.clone() for t in (C.k, C.v, C.acc, C.pos))
    got_k = C.kd.cpu()
    th = L.theta(rot) if rot else None
    for i, m in enumerate(new):
        if m == 0 or not 0 <= C.slots[i] < C.n_slots:
            continue
        rows = np.arange(held[i], held[i] + m)
        at = slice(cu[i], cu[i] + m)
        p = rows if pos is None else pos[at]

        def turned(x, heads):
            x = f64(x[at]).reshape(m, heads, d)
            return L.rotate(x, p, th, rot, inter) if rot else (x, np.zeros(x.shape))

        pg = C.table[C.slots[i]][rows // page].astype(np.int64)
        there = (pg >= 0) & (pg < C.n_pages)
        ref, err = turned(k, hk)
        got = f64(got_k[pg[there], :, (rows % page)[there]])
        assert not (np.abs(got - ref[there]) > (err + (np.abs(ref) + err) * L.ROUND[io])[there] * (rot > 0)).any(), i
        wk[pg[there], :, (rows % page)[there]] = got_k[pg[there], :, (rows % page)[there]]
        wv[pg[there], :, (rows % page)[there]] = v[at].reshape(m, hk, d)[torch.from_numpy(there)]
        if C.acc is not None:
            wacc[pg[there], :, (rows % page)[there]] = 0.0
            new_pos = torch.from_numpy(p[there].astype(np.int32))[:, None]
            wpos[pg[there], :, (rows % page)[there]] = new_pos.expand(-1, hk)
        if with_q:
            ref, err = turned(q, H)
            got = f64(od[at]).reshape(m, H, d)
            assert not (np.abs(got - ref) > (err + (np.abs(ref) + err) * L.ROUND[io]) * (rot > 0)).any(), i
            obuf[at, off:off + H * d] = before[at, off:off + H * d]
    assert same(C.kd, wk) and same(C.vd, wv)
    assert C.acc is None or (same(C.accd, wacc) and same(C.posd, wpos))
    assert torch.equal(obuf, before)


def test_in_place_and_bad_lengths():
    """Queries turned in place; a slot whose lens is shorter than the new tokens, negative or beyond its table is
    skipped."""
    torch = torch_cuda()
    g = lib()
    say("append in place")
    rng = np.random.default_rng(3)
    C = Cache(rng, [20, 20, 20, 20], 2, 64, 16, "bf16")
    C.lens[C.slots[1]], C.lens[C.slots[2]], C.lens[C.slots[3]] = 2, -3, C.max_pages * 16 + 1
    C.lensd = up(C.lens)
    new = [3, 3, 3, 3]
    cu = np.array([0, 3, 6, 9, 12], np.int32)
    q, k, v = rand(rng, (12, 4 * 64), "bf16"), rand(rng, (12, 128), "bf16").cuda(), rand(rng, (12, 128), "bf16").cuda()
    qd = q.cuda()
    rope = g.RopeDesc(d=64)
    g.gdnq_kv_append(g.AttnDesc(H=4, hk=2, d=64, page=16), rope, table_of(rope), C.kv(), qd, qd, k, v, None, C.slotsd,
                     up(cu), 4, 12)
    ref, err = L.rotate(f64(q[:3]).reshape(3, 4, 64), np.arange(17, 20), L.theta(64), 64)
    assert not (np.abs(f64(qd[:3]).reshape(ref.shape) - ref) > err + (np.abs(ref) + err) * L.ROUND["bf16"]).any()
    assert torch.equal(qd[3:].cpu(), q[3:])
    want = C.v.clone()
    pg, off = C.where(0, 17, 20)
    want[pg, :, off] = v[:3].cpu().reshape(3, 2, 64)
    assert same(C.vd, want) and sum(new) == 12


@pytest.mark.parametrize("off", [0, 3])
def test_long_calls(off):
    """A call whose rows go past the caches, several tokens to a workgroup, gives
    what calls on its sequences give, bit for bit."""
    torch = torch_cuda()
    g = lib()
    say("append, long call", off)
    new, H, hk, d, page = [2000, 1, 0, 1501, 6, 700], 32, 8, 128, 16
    rng = np.random.default_rng(23)
    got = []
    T = sum(new)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(T, (H + 2 * hk) * d + off, generator=gen, device="cuda").bfloat16()[:, off:]
    assert 2 * x.numel() * 2 > 64 << 20
    q, k, v = x[:, :H * d], x[:, H * d:(H + hk) * d], x[:, (H + hk) * d:]
    rope = g.RopeDesc(d=d, rot=92, flags=g.ROPE_INTERLEAVED)
    desc, freqs = g.AttnDesc(H=H, hk=hk, d=d, page=page), table_of(rope)
    C = Cache(rng, [m + 5 for m in new], hk, d, page, "bf16", fill=0.0)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    for whole in (True, False):
        kk, vv, acc, pos = C.kd.clone(), C.vd.clone(), C.accd.clone(), C.posd.clone()
        o = torch.zeros_like(q)
        kv = g.Kv(kk, vv, C.tabled, C.lensd, acc, pos)
        if whole:
            g.gdnq_kv_append(desc, rope, freqs, kv, q, o, k, v, None, C.slotsd, up(cu), len(new), T)
        else:
            for i, m in enumerate(new):
                at = slice(cu[i], cu[i] + m)
                slot = up(C.slots[i:i + 1])
                if m:   # up to 900 tokens: one to a workgroup; the lens of a part count what lies behind it
                    lens = C.lens.copy()
                    for lo in range(0, m, 900):
                        n = min(900, m - lo)
                        lens[C.slots[i]] = C.lens[C.slots[i]] - (m - lo - n)
                        part = slice(at.start + lo, at.start + lo + n)
                        kv = g.Kv(kk, vv, C.tabled, up(lens), acc, pos)
                        g.gdnq_kv_append(desc, rope, freqs, kv, q[part], o[part], k[part], v[part], None, slot,
                                         up(np.array([0, n], np.int32)), 1, n)
        got.append((kk, vv, acc, pos, o))
    assert all(same(a, b) for a, b in zip(*got))
