"""Measured cases of the operators of a softmax attention layer beside the
recurrent ones: rotary positions, storing into a paged cache of keys and values,
the attention of one new token over it, and eviction from it by accumulated
attention weight.

``run`` computes a case's operator in elementary torch operations, or with
``own`` set calls the library.  ``exact`` computes it in 64 bits, entry by entry.

A case's kind says which call it is:
  rope    gdnq_rope: every head of every token row turned by its position
  append  gdnq_kv_append: the queries of new tokens turned, their keys turned and
          stored with their values behind the rows that each request's cache holds
  attn    gdnq_attn_step: one new token of each running request over its cache
  evict   gdnq_kv_evict: the rows of least accumulated weight leave each cache
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # decode of three requests: launch latency counts; the query and key heads of a fused projection,
        # a quarter of a wide head turns
        dict(name="rope token x3", kind="rope", io="bf16", rows=3, H=18, d=256, rot=64, inter=False, inverse=False,
             scaling="plain", far=40000),
        # prefill: query and key heads of long prompts at positions up to a million, scaled by a ramp over the pairs
        dict(name="rope prompts 32768", kind="rope", io="bf16", rows=32768, H=40, d=128, rot=128, inter=False,
             inverse=False, scaling="index", far=1000000),
        # the gradient of a batch's rotation in fp32: interleaved pairs, three quarters of the head
        dict(name="rope gradient 8191", kind="rope", io="f32", rows=8191, H=24, d=128, rot=96, inter=True, inverse=True,
             scaling="turns", far=131072),
        # decode of one request: its queries, key and value
        dict(name="append token x1", kind="append", io="bf16", H=32, hk=8, d=128, page=16, rot=128, inter=False,
             packed=False, n=1, tokens=1, tail=0, held=5000, lens=1),
        # prefill of a mixed batch of prompts, some of them continued
        dict(name="append prompts 20011", kind="append", io="bf16", H=32, hk=8, d=128, page=64, rot=64, inter=True,
             packed=True, n=13, tokens=20011, tail=53, held=3000, lens=2),
        # decode of one short request: wide heads, eight query heads to a cache head
        dict(name="attention x1 of 700", kind="attn", io="bf16", H=16, hk=2, d=256, page=16, n=1, least=700, most=700,
             window=0, sums=False, lens=3),
        # decode of one long request: few rows, a long axis
        dict(name="attention x1 of 131071", kind="attn", io="bf16", H=32, hk=8, d=128, page=64, n=1, least=131071,
             most=131071, window=0, sums=False, lens=4),
        # decode of a serving batch of very different lengths
        dict(name="attention x64 to 32768", kind="attn", io="bf16", H=32, hk=8, d=128, page=64, n=64, least=512,
             most=32768, window=0, sums=False, lens=5),
        # decode of a batch with bounded caches: the weights are summed up for the eviction
        dict(name="attention sums x192 to 2100", kind="attn", io="bf16", H=32, hk=4, d=128, page=32, n=192, least=1500,
             most=2100, window=0, sums=True, lens=6),
        # fp32, a window of rows, three query heads of 64 channels to a cache head
        dict(name="attention window x24 f32", kind="attn", io="f32", H=24, hk=8, d=64, page=16, n=24, least=900,
             most=6000, window=1500, sums=False, lens=7),
        # a decode step of a batch with bounded caches: one row of each leaves
        dict(name="evict one of x64", kind="evict", io="bf16", H=32, hk=8, d=128, page=32, n=64, budget=2048,
             least=2049, most=2049, sink=4, recent=128, lens=8),
        # behind the prompts: each cache is cut down to its bound
        dict(name="evict prompts x8", kind="evict", io="bf16", H=32, hk=8, d=128, page=64, n=8, budget=2048,
             least=6000, most=20000, sink=4, recent=256, lens=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attn", "attn", "evict"])
    c = dict(kind=kind, io=rng.choice(["bf16", "bf16", "f32"]), d=rng.choice([64, 128, 128, 256]))
    if kind != "rope":
        c["hk"] = rng.choice([1, 2, 3, 4, 8])
        c["H"] = c["hk"] * rng.choice([1, 2, 3, 4, 5, 8, 16] if c["hk"] < 8 else [1, 2, 4, 5])
        c["page"] = rng.choice([8, 16, 32, 64, 128])
        c["lens"] = rng.randrange(1 << 20)
    if kind in ("rope", "append"):
        if kind == "rope":
            c["d"] = rng.choice([64, 128, 256, 2 * rng.randrange(8, 160)])
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 4 * 2, 2 * rng.randrange(1, c["d"] // 2 + 1)])
        c["inter"] = rng.random() < 0.5
    if kind == "rope":
        c.update(rows=_log(rng, 1, 16000), H=rng.randrange(1, 41), inverse=rng.random() < 0.3,
                 scaling=rng.choice(["plain", "linear", "base", "turns", "index"]), far=_log(rng, 100, 1000000))
    if kind == "append":
        c["packed"] = rng.random() < 0.6
        c["n"] = _log(rng, 1, 40 if c["packed"] else 700)
        c["tokens"] = c["n"] if not c["packed"] else _log(rng, c["n"], 14000)
        c["tail"] = rng.randrange(0, 60) if c["packed"] else 0
        c["held"] = _log(rng, 1, 3000)
    if kind == "attn":
        c["n"] = _log(rng, 1, 256)
        # rows of K and V up to about 1 GB in all, the padded batch of the plain form within 4 GB
        room = 1 << 29
        most = max(8, room // (c["n"] * c["hk"] * c["d"] * (2 if c["io"] == "bf16" else 4)))
        c["most"] = _log(rng, 4, min(most, 150000))
        c["least"] = _log(rng, 1, c["most"])
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, c["most"])])
        c["sums"] = rng.random() < 0.4
    if kind == "evict":
        c["n"] = _log(rng, 1, 64)
        most = min(20000, (1 << 26) // (c["n"] * c["hk"] * c["d"]))
        c["budget"] = _log(rng, 40, max(50, most // 2))
        c["most"] = c["budget"] + _log(rng, 1, max(2, most - c["budget"]))
        c["least"] = rng.choice([c["most"], c["most"], max(1, c["budget"] - 20)])
        c["sink"] = rng.choice([0, 4, 16])
        c["recent"] = rng.choice([0, 1, 8, c["budget"] // 4])
    return c


def _lengths(case):
    """The rows that each entry's cache holds (attention, eviction): between least and most, more short ones than
    long ones, the longest among them (attention: one of none and one of one row where there are several).  The
    tokens of each prompt (append), one of them zero and one a single token where there are several."""
    r = random.Random(case["lens"])
    n = case["n"]
    if case["kind"] != "append":
        v = [_log(r, case["least"], case["most"]) for _ in range(n)]
        if case["kind"] == "attn" and n >= 6:
            v[n // 2], v[n // 3] = 0, 1
        v[-1] = case["most"]
        return v
    if not case["packed"]:
        return [1] * n
    w = [math.exp(r.gauss(0.0, 1.0)) for _ in range(n)]
    if n >= 6:
        w[n // 2] = w[n // 3] = 0.0
    v = [int(case["tokens"] * x / sum(w)) for x in w]
    if n >= 6:
        v[n // 3] = 1
    v[0] += case["tokens"] - sum(v)
    return v if v[0] >= 0 else [case["tokens"]] + [0] * (n - 1)


def _attended(case):
    w = case["window"]
    return [min(x, w) if w else x for x in _lengths(case)]


def _item(case):
    return 2 if case["io"] == "bf16" else 4


def work(case):
    k, it = case["kind"], _item(case)
    if k == "rope":
        e = case["rows"] * case["H"] * case["d"]
        return {"bytes": 2 * it * e + 4 * case["rows"], "flops": 3 * case["rows"] * case["H"] * case["rot"]}
    if k == "append":
        h = case["H"] + case["hk"]
        return {"bytes": case["tokens"] * (2 * it * case["d"] * (h + case["hk"]) + 4 + 8 * case["hk"]),
                "flops": 3 * case["tokens"] * h * case["rot"]}
    if k == "attn":
        rows, q = sum(_attended(case)), case["n"] * case["H"] * case["d"]
        return {"bytes": rows * case["hk"] * (2 * it * case["d"] + 8 * case["sums"]) + 2 * it * q,
                "flops": 4 * rows * case["H"] * case["d"]}
    b = 0.0
    for n in _lengths(case):
        if n > case["budget"]:   # the kept rows behind the budget: the recent ones, and a share of the others
            t = n - case["budget"]
            r = min(case["recent"], t)
            left = n - case["sink"] - case["recent"]
            moved = r + (t - r) * max(0, case["budget"] - case["sink"] - case["recent"]) / max(1, left)
            b += case["hk"] * (8 * n + 2 * moved * (2 * it * case["d"] + 8))
    return {"bytes": max(b, 8.0), "flops": 0}


# ------------------------------------------------------------------ inputs
def _io(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


BASE, ORIG, FACTOR = 500000.0, 4096.0, 16.0


def _scaling(case):
    """The scaling's numbers by name: how long the contexts were that the frequencies come from, by how much they
    grow, and between how many turns over them the ramps lie."""
    return dict(plain=dict(base=10000.0), linear=dict(base=10000.0, factor=4.0), base=dict(base=10000.0, factor=8.0),
                turns=dict(base=BASE, factor=8.0, orig_len=8192.0, lo=1.0, hi=4.0),
                index=dict(base=BASE, factor=FACTOR, orig_len=ORIG, lo=1.0, hi=32.0))[case.get("scaling", "plain")]


def _amp(case):
    return 0.1 * math.log(FACTOR) + 1.0 if case.get("scaling") == "index" else 1.0


def _theta(case):
    """Angles per position of the pairs, in Python's 64 bits."""
    z, rot, kind = _scaling(case), case["rot"], case.get("scaling", "plain")
    base, f = z["base"], z.get("factor", 1.0)
    if kind == "base" and rot > 2:
        base *= f ** (rot / (rot - 2))
    out = []
    if kind == "index":
        at = [rot / 2 * math.log(ORIG / (2 * math.pi * t)) / math.log(base) for t in (z["hi"], z["lo"])]
        i0, i1 = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    for i in range(rot // 2):
        t = base ** (-2.0 * i / rot)
        keep = 1.0
        if kind == "linear":
            keep = 0.0
        elif kind == "turns":
            keep = min(1.0, max(0.0, (z["orig_len"] * t / (2 * math.pi) - z["lo"]) / (z["hi"] - z["lo"])))
        elif kind == "index":
            keep = 1.0 - min(1.0, max(0.0, (i - i0) / ((i1 - i0) or 0.001)))
        out.append(t * (keep + (1.0 - keep) / f) if kind != "base" else t)
    return out


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = random.Random(seed)
    dt = _io(case)

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    k = case["kind"]
    s = {"case": case, "kind": k}
    if k in ("rope", "append"):
        s["theta"] = torch.tensor(_theta(case), dtype=torch.float64, device=dev)
    if k == "rope":
        n = case["rows"]
        s["x"] = normal(n, case["H"] * case["d"])
        s["y"] = torch.empty_like(s["x"])
        start = rnd.randrange(case["far"])
        s["pos"] = ints([(start + 7 * i) % case["far"] for i in range(n)])
        if own:
            _handles(s)
        return s
    H, hk, d, page = case["H"], case["hk"], case["d"], case["page"]
    lens = _lengths(case)
    n = len(lens)
    if k == "append":
        cu = [0]
        for m in lens:
            cu.append(cu[-1] + m)
        T = case["tokens"] + case["tail"]
        before = random.Random(case["lens"] + 1)
        held = [before.randrange(case["held"] + 1) for _ in lens]
        s.update(T=T, total=cu[-1], cu=ints(cu), new=lens)
        lens = [a + b for a, b in zip(held, lens)]
        s["q"], s["k_new"], s["v_new"] = normal(T, H * d), normal(T, hk * d), normal(T, hk * d)
        s["q_out"] = torch.full((T, H * d), 0.5, dtype=dt, device=dev)
    # a pool with a few pages and slots more than needed; the entries' slots and pages in no order, and a page
    # that no entry holds where a table has none
    n_slots, most = n + 3, max(lens)
    max_pages = -(-most // page)
    need = [-(-m // page) for m in lens]
    n_pages = sum(need) + 5
    order = list(range(n_pages))
    rnd.shuffle(order)
    slots = rnd.sample(range(n_slots), n)
    table, slot_lens, at = [[order[-1]] * max_pages for _ in range(n_slots)], [0] * n_slots, 0
    for i, m in enumerate(need):
        table[slots[i]][:m] = order[at:at + m]
        slot_lens[slots[i]] = lens[i]
        at += m
    s.update(n=n, lens_host=lens, slots_host=slots, most=most, n_pages=n_pages, slots=ints(slots), table=ints(table),
             lens=ints(slot_lens))
    s["k"], s["v"] = normal(n_pages, hk, page, d), normal(n_pages, hk, page, d)
    s["acc"] = s["pos"] = None
    if k == "append":
        s["acc"] = torch.full((n_pages, hk, page), 0.25, device=dev)
        s["pos"] = torch.full((n_pages, hk, page), -1, dtype=torch.int32, device=dev)
    if k == "attn":
        s["q"] = normal(n, H * d, scale=2.0)   # a few rows of many hold most of the weight
        s["o"] = torch.empty(n, H * d, dtype=dt, device=dev)
        if case["sums"]:
            s["acc"] = torch.rand(n_pages, hk, page, generator=g, device=dev)
    if k == "evict":
        # sums as decoding leaves them, a share of them at zero; every cache holds its newest tokens at its end
        u = torch.rand(n_pages, hk, page, generator=g, device=dev)
        s["acc0"] = torch.where(u < 0.05, torch.zeros_like(u), u ** 4)
        s["pos0"] = torch.zeros(n_pages, hk, page, dtype=torch.int32, device=dev)
        pages = s["table"][s["slots"].long()].long()
        row = torch.arange(max_pages * page, dtype=torch.int32, device=dev).reshape(1, max_pages, 1, page)
        ln = torch.tensor(lens, dtype=torch.int32, device=dev).reshape(n, 1, 1, 1)
        seen = ln + 1000                       # tokens seen: gaps between the older rows
        older = row.long() * (seen - case["recent"] - 1) // torch.clamp(ln - case["recent"], min=1)
        p = torch.where(row >= ln - case["recent"], row + 1000, older.int()).expand(n, max_pages, hk, page)
        held = torch.arange(max_pages, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
        s["pos0"][pages[held]] = p[held]
        s["acc"], s["pos"] = s["acc0"].clone(), s["pos0"].clone()
    if own:
        _handles(s)
    return s


def _handles(s):
    """The descriptors, the frequencies, the cache and the workspace that a program keeps for a layer."""
    import recurrent_state_quantization_amd as lib

    c, k = s["case"], s["kind"]
    io = lib.IO_BF16 if c["io"] == "bf16" else lib.IO_F32
    s["lib"] = lib
    if k in ("rope", "append"):
        flags = (lib.ROPE_INTERLEAVED if c["inter"] else 0) | (lib.ROPE_INVERSE if c.get("inverse") else 0)
        s["rope"] = lib.RopeDesc(d=c["d"], rot=c["rot"], io_dtype=io, flags=flags, amp=_amp(c)).c()
        kind = dict(plain=lib.ROPE_PLAIN, linear=lib.ROPE_LINEAR, base=lib.ROPE_BASE, turns=lib.ROPE_RAMP_TURNS,
                    index=lib.ROPE_RAMP_INDEX)[c.get("scaling", "plain")]
        s["freqs"] = lib.gdnq_rope_table(s["rope"], lib.RopeFreqs(kind=kind, **_scaling(c))).cuda()
    if k == "rope":
        return
    s["desc"] = lib.AttnDesc(H=c["H"], hk=c["hk"], d=c["d"], io_dtype=io, page=c["page"],
                             window=c.get("window", 0)).c()
    s["kv"] = lib.Kv(k=s["k"], v=s["v"], table=s["table"], lens=s["lens"], acc=s["acc"], pos=s["pos"]).c(s["desc"])
    s["ws"] = None
    if k == "append":
        return
    nb = lib.gdnq_attn_workspace(s["desc"], s["kv"], s["n"]) if k == "attn" else \
        lib.gdnq_kv_evict_workspace(s["desc"], s["kv"], c["budget"], s["n"])
    s["ws"] = torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None


# --------------------------------------------------------------- the calls
def run(s):
    if s["kind"] == "evict":
        # decoding goes on between two evictions; here the first sums are put back
        s["acc"].copy_(s["acc0"])
        s["pos"].copy_(s["pos0"])
    return (_run_own if own else _PLAIN[s["kind"]])(s)


def _run_own(s):
    lib, k, c = s["lib"], s["kind"], s["case"]
    if k == "rope":
        lib.gdnq_rope(s["rope"], s["freqs"], s["x"], s["pos"], s["y"], c["rows"], c["H"])
        return {"y": s["y"]}
    if k == "append":
        lib.gdnq_kv_append(s["desc"], s["rope"], s["freqs"], s["kv"], s["q"], s["q_out"], s["k_new"], s["v_new"], None,
                           s["slots"], s["cu"] if c["packed"] else None, s["n"], s["T"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"], "acc": s["acc"], "pos": s["pos"]}
    if k == "attn":
        lib.gdnq_attn_step(s["desc"], s["kv"], s["q"], s["o"], s["slots"], s["n"], s["ws"])
        return {"o": s["o"], "acc": s["acc"]} if c["sums"] else {"o": s["o"]}
    lib.gdnq_kv_evict(s["desc"], s["kv"], c["budget"], c["sink"], c["recent"], s["slots"], s["n"], s["ws"])
    return {"k": s["k"], "v": s["v"], "acc": s["acc"], "pos": s["pos"]}


# --------------------------------------------------------- the plain forms
def _rotate(s, x, pos, heads):
    """x [rows, heads*d] turned by pos [rows], in fp32; the angles in 64 bits."""
    c = s["case"]
    d, rot = c["d"], c["rot"]
    x = x.float().reshape(-1, heads, d)
    a = pos.double()[:, None] * s["theta"]
    cos, sin = (torch.cos(a) * _amp(c)).float()[:, None], (torch.sin(a) * _amp(c)).float()[:, None]
    if c.get("inverse"):
        sin = -sin
    if c["inter"]:
        u, w = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).reshape(-1, heads, rot)
    else:
        u, w = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    return torch.cat([y, x[..., rot:]], -1).reshape(-1, heads * d)


def _plain_rope(s):
    s["y"].copy_(_rotate(s, s["x"], s["pos"], s["case"]["H"]))
    return {"y": s["y"]}


def _plain_append(s):
    c, total = s["case"], s["total"]
    hk, d, page = c["hk"], c["d"], c["page"]
    t = torch.arange(total, device=s["q"].device)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    slot = s["slots"].long()[seq]
    row = s["lens"].long()[slot] - (cu[seq + 1] - t)
    pg, off = s["table"].long()[slot, row // page], row % page
    s["q_out"][:total] = _rotate(s, s["q"][:total], row, c["H"]).to(s["q"].dtype)
    s["k"][pg, :, off] = _rotate(s, s["k_new"][:total], row, hk).reshape(total, hk, d).to(s["k"].dtype)
    s["v"][pg, :, off] = s["v_new"][:total].reshape(total, hk, d)
    s["acc"][pg, :, off] = 0.0
    s["pos"][pg, :, off] = row.int()[:, None].expand(total, hk)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "acc": s["acc"], "pos": s["pos"]}


def _rows_of(s):
    """Pages [n, max_pages], row numbers [R] and which of them each entry holds [n, R]."""
    slot = s["slots"].long()
    pages = s["table"].long()[slot]
    row = torch.arange(pages.shape[1] * s["case"]["page"], device=pages.device)
    return pages, row, s["lens"].long()[slot]


def _plain_attn(s):
    c, n = s["case"], s["n"]
    H, hk, d, page = c["H"], c["hk"], c["d"], c["page"]
    pages, row, ln = _rows_of(s)
    R = row.shape[0]

    def rows(cache):   # [n, hk, R, d]
        return cache[pages].transpose(1, 2).reshape(n, hk, R, d).float()

    q = s["q"].float().reshape(n, hk, H // hk, d)
    sc = torch.matmul(q, rows(s["k"]).transpose(-1, -2)) / math.sqrt(d)
    live = row[None] < ln[:, None]
    if c["window"]:
        live = live & (row[None] >= ln[:, None] - c["window"])
    sc = torch.where(live[:, None, None], sc, torch.full_like(sc, -math.inf))
    p = torch.exp(sc - torch.clamp(sc.amax(-1, keepdim=True), min=-3e38))
    p = p / torch.clamp(p.sum(-1, keepdim=True), min=1e-38)   # no rows: no weights, an output of zeros
    s["o"].copy_(torch.matmul(p, rows(s["v"])).reshape(n, H * d))
    if not c["sums"]:
        return {"o": s["o"]}
    w = p.sum(2).reshape(n, hk, R // page, page).transpose(1, 2)     # [n, pages, hk, page]
    has = (torch.arange(R // page, device=row.device)[None] * page < ln[:, None])[..., None, None]
    s["acc"].index_put_((pages,), torch.where(has, w, torch.zeros_like(w)), accumulate=True)
    return {"o": s["o"], "acc": s["acc"]}


def _plain_evict(s):
    c, n = s["case"], s["n"]
    hk, page, budget = c["hk"], c["page"], c["budget"]
    pages, row, ln = _rows_of(s)
    R = row.shape[0]
    head = torch.arange(hk, device=row.device)

    def rows(cache):   # [n, hk, R]
        return cache[pages].transpose(1, 2).reshape(n, hk, R)

    live = (row[None] < ln[:, None])[:, None]
    pos = torch.where(live, rows(s["pos"]), torch.full_like(row.int(), -1))
    safe = (pos < c["sink"]) | (pos > pos.amax(-1, keepdim=True) - c["recent"])
    key = torch.where(safe, torch.full_like(rows(s["acc"]), 3e38), rows(s["acc"]))
    key = torch.where(live, key, torch.full_like(key, math.inf))
    rank = torch.argsort(torch.argsort(key, dim=-1, stable=True), dim=-1)   # ties: the lower row first
    gone = rank < torch.clamp(ln - budget, min=0)[:, None, None]
    big = 2 * R
    hole = torch.sort(torch.where(gone & (row < budget), row, big), -1)[0][..., :max(R - budget, 0)]
    kept = torch.sort(torch.where(live & ~gone & (row >= budget), row, big), -1)[0][..., :hole.shape[-1]]
    # no hole, no move: the row behind the budget stays what it is
    dst, src = torch.where(hole < big, hole, min(budget, R - 1)), torch.where(kept < big, kept, min(budget, R - 1))
    at = torch.arange(n, device=row.device)[:, None, None]

    def place(r):
        return pages[at, r // page], head[None, :, None], r % page

    src, dst = place(src), place(dst)
    s["k"][dst], s["v"][dst] = s["k"][src], s["v"][src]
    s["acc"][dst], s["pos"][dst] = s["acc"][src], s["pos"][src]
    return {"k": s["k"], "v": s["v"], "acc": s["acc"], "pos": s["pos"]}


_PLAIN = {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "evict": _plain_evict}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["kind"]](s, case)


def _theta64(c, dev):
    """The pairs' angles per position, from the definition of each scaling."""
    z, rot, kind = _scaling(c), c["rot"], c.get("scaling", "plain")
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    base, f = z["base"], z.get("factor", 1.0)
    t = torch.exp(-2.0 * i / rot * math.log(base))
    if kind == "plain":
        return t
    if kind == "linear":
        return t / f
    if kind == "base":   # the last pair slower by the factor, the first as it was
        return t * torch.exp(-math.log(f) * i / (rot // 2 - 1)) if rot > 2 else t
    if kind == "turns":
        keep = ((z["orig_len"] * t / (2 * math.pi) - z["lo"]) / (z["hi"] - z["lo"])).clamp(0, 1)
    else:
        def pair(turns):   # the pair that makes so many turns over the old length
            return rot * math.log(z["orig_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(0, math.floor(pair(z["hi"]))), min(rot - 1, math.ceil(pair(z["lo"])))
        keep = 1 - ((i - first) / (last - first if last != first else 0.001)).clamp(0, 1)
    return keep * t + (1 - keep) * t / f


def _turn64(c, x, pos, heads):
    """Every pair as a complex number times e^{i angle}."""
    d, rot = c["d"], c["rot"]
    x = x.double().reshape(-1, heads, d).clone()
    a = pos.double()[:, None, None] * _theta64(c, x.device)
    one = torch.polar(torch.full_like(a, _amp(c)), -a if c.get("inverse") else a)
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if c["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., lo], x[..., hi]) * one
    x[..., lo], x[..., hi] = z.real, z.imag
    return x.reshape(-1, heads * d)


def _exact_rope(s, c):
    return {"y": _turn64(c, s["x"], s["pos"], c["H"])}


def _table64(s, i):
    """The pages of entry i's rows and their places in them."""
    c, n = s["case"], s["lens_host"][i]
    r = torch.arange(n, device=s["k"].device)
    return s["table"][s["slots_host"][i]].long()[r // c["page"]], r % c["page"]


def _exact_append(s, c):
    q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
    acc, pos = s["acc"].double(), s["pos"].clone()
    at = 0
    for i, m in enumerate(s["new"]):
        if m == 0:
            continue
        n = s["lens_host"][i]
        p = torch.arange(n - m, n, device=k.device)
        pg, off = (t[n - m:] for t in _table64(s, i))
        q[at:at + m] = _turn64(c, s["q"][at:at + m], p, c["H"])
        k[pg, :, off] = _turn64(c, s["k_new"][at:at + m], p, c["hk"]).reshape(m, c["hk"], -1)
        v[pg, :, off] = s["v_new"][at:at + m].double().reshape(m, c["hk"], -1)
        acc[pg, :, off] = 0
        pos[pg, :, off] = p.int()[:, None]
        at += m
    return {"q": q, "k": k, "v": v, "acc": acc, "pos": pos}


def _exact_attn(s, c):
    H, hk, d = c["H"], c["hk"], c["d"]
    o = torch.zeros(s["n"], H, d, dtype=torch.float64, device=s["q"].device)
    acc = s["acc"].double() if c["sums"] else None
    for i, n in enumerate(s["lens_host"]):
        lo = max(0, n - c["window"]) if c["window"] else 0
        pg, off = (t[lo:] for t in _table64(s, i))
        if n == 0:
            continue
        for h in range(hk):
            g = slice(h * (H // hk), (h + 1) * (H // hk))
            q = s["q"][i].double().reshape(H, d)[g]
            w = torch.softmax(q @ s["k"][pg, h, off].double().T.contiguous() / d ** 0.5, -1)
            o[i, g] = w @ s["v"][pg, h, off].double()
            if acc is not None:
                acc[pg, h, off] += w.sum(0)
    out = {"o": o.reshape(s["n"], H * d)}
    return out if acc is None else {**out, "acc": acc}


def _exact_evict(s, c):
    k, v, acc, pos = s["k"].clone(), s["v"].clone(), s["acc0"].clone(), s["pos0"].clone()
    for i, n in enumerate(s["lens_host"]):
        if n <= c["budget"]:
            continue
        pg, off = _table64(s, i)
        for h in range(c["hk"]):
            a, p = acc[pg, h, off].double(), pos[pg, h, off]
            a[(p < c["sink"]) | (p > p.max() - c["recent"])] = math.inf
            gone = torch.zeros(n, dtype=torch.bool, device=a.device)
            gone[torch.sort(a, stable=True)[1][:n - c["budget"]]] = True
            hole = torch.nonzero(gone[:c["budget"]])[:, 0]
            kept = torch.nonzero(~gone[c["budget"]:])[:, 0] + c["budget"]
            for t in (k, v, acc, pos):
                t[pg[hole], h, off[hole]] = t[pg[kept], h, off[kept]]
    return {"k": k.double(), "v": v.double(), "acc": acc.double(), "pos": pos}


_EXACT = {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn, "evict": _exact_evict}
