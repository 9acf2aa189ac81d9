"""The C ABI of include/gdnq_attn.h without a GPU: exports, struct layouts, the
refusal of every invalid argument on the host, and the table of frequencies.
Device pointers are fake aligned addresses: a rejected call never dereferences
them."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from tests import _attn as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdnq_attn.h")
NAMES = ["gdnq_attn_step", "gdnq_attn_workspace", "gdnq_kv_append", "gdnq_kv_evict", "gdnq_kv_evict_workspace",
         "gdnq_rope", "gdnq_rope_table"]
BASE = 1 << 40


@pytest.fixture(scope="module")
def g():
    import recurrent_state_quantization_amd as g
    return g


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_every_declared_symbol_is_exported(g):
    assert sorted(re.findall(r"^int\s+(\w+)\s*\(", _text(), flags=re.M)) == NAMES
    out = subprocess.run(["nm", "-D", "--defined-only", g.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert not [n for n in NAMES if n not in exported]
    assert not [n for n in NAMES if not hasattr(g, n)]


@pytest.mark.parametrize("name,mirror", [("gdnq_rope_desc", "_RopeDesc"), ("gdnq_rope_freqs", "_RopeFreqs"),
                                         ("gdnq_attn_desc", "_AttnDesc"), ("gdnq_kv", "_Kv")])
def test_struct_layouts_match_header(g, name, mirror):
    from recurrent_state_quantization_amd import attn
    body = [b for b, n in re.findall(r"typedef struct \{([^}]*)\} (\w+);", _text()) if n == name][0]
    fields = [re.sub(r"\W", "", f.split()[-1]) for d in body.split(";") for f in d.split(",") if f.strip()]
    assert fields == [f[0] for f in getattr(attn, mirror)._fields_]


def test_values_match_header(g):
    text = open(HEADER).read()
    for k in ("INTERLEAVED", "INVERSE"):
        assert int(re.search(rf"#define GDNQ_ROPE_{k} (\d+)u", text).group(1)) == getattr(g, f"ROPE_{k}")
    for k in ("PLAIN", "LINEAR", "BASE", "RAMP_TURNS", "RAMP_INDEX"):
        assert int(re.search(rf"GDNQ_ROPE_{k} = (\d+)", text).group(1)) == getattr(g, f"ROPE_{k}")


def test_header_is_c(tmp_path):
    f = tmp_path / "t.c"
    f.write_text('#include "gdnq_attn.h"\n#include "gdnq_layer.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER), str(f)],
                   check=True)


# ------------------------------------------------------------ frequencies
KINDS = [("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
         ("turns", dict(base=5e5, factor=8.0, orig_len=8192.0, lo=1.0, hi=4.0)),
         ("index", dict(base=5e5, factor=16.0, orig_len=4096.0, lo=1.0, hi=32.0)),
         ("index", dict(base=2.0, factor=2.0, orig_len=1e9, lo=1.0, hi=32.0)),
         ("index", dict(base=1e30, factor=2.0, orig_len=64.0, lo=1.0, hi=1.01))]


@pytest.mark.parametrize("kind,kw", KINDS, ids=[k + str(i) for i, (k, _) in enumerate(KINDS)])
@pytest.mark.parametrize("rot", [2, 6, 64, 128, 1024])
@pytest.mark.parametrize("div", [False, True])
def test_table(g, kind, kw, rot, div):
    divisors = list(np.linspace(1.0, 9.7, rot // 2)) if div else None
    code = dict(plain=g.ROPE_PLAIN, linear=g.ROPE_LINEAR, base=g.ROPE_BASE, turns=g.ROPE_RAMP_TURNS,
                index=g.ROPE_RAMP_INDEX)[kind]
    got = g.gdnq_rope_table(g.RopeDesc(d=1024, rot=rot), g.RopeFreqs(kind=code, divisors=divisors, **kw))
    got = got.numpy().view(np.uint64).astype(L.LD)
    want = (L.theta(rot, kind, divisors=divisors, **kw) / L.PI2 % 1) * L.LD(2) ** 64
    # both in long double: a few units of its 2^-64 from the power and the products, and the table's half
    assert np.abs(got - want).max() <= 64
    if kind == "plain" and not div:
        assert got[0] == round(2 ** 64 / (2 * np.pi), -3) or abs(float(got[0]) * 2 * np.pi / 2 ** 64 - 1) < 1e-15


@pytest.mark.parametrize("kw,code,msg", [
    (dict(desc=dict(d=3)), 2, "d must"),
    (dict(desc=dict(d=0)), 2, "d must"),
    (dict(desc=dict(d=1026)), 2, "d must"),
    (dict(desc=dict(rot=7)), 1, "rot must"),
    (dict(desc=dict(rot=66)), 1, "rot must"),
    (dict(desc=dict(rot=-2)), 1, "rot must"),
    (dict(desc=dict(io_dtype=2)), 1, "io_dtype"),
    (dict(desc=dict(flags=4)), 1, "flag"),
    (dict(desc=dict(amp=0.0)), 1, "amp"),
    (dict(desc=dict(amp=float("nan"))), 1, "amp"),
    (dict(desc=dict(amp=float("inf"))), 1, "amp"),
    (dict(kind=5), 1, "kind"),
    (dict(kind=-1), 1, "kind"),
    (dict(base=1.0), 1, "base"),
    (dict(base=float("inf")), 1, "base"),
    (dict(base=float("nan")), 1, "base"),
    (dict(kind=1, factor=0.0), 1, "factor"),
    (dict(kind=3, factor=2.0), 1, "orig_len"),
    (dict(kind=3, factor=2.0, orig_len=10.0, lo=2.0, hi=2.0), 1, "lo < hi"),
    (dict(kind=4, factor=2.0, orig_len=10.0, lo=0.0, hi=2.0), 1, "lo < hi"),
    (dict(divisors=[1.0] * 31 + [0.0]), 1, "divisors[31]"),
    (dict(divisors=[1.0] * 31), 1, "divisors has 31"),
])
def test_table_refusals(g, kw, code, msg):
    desc = g.RopeDesc(**{"d": 64, **kw.pop("desc", {})})
    with pytest.raises(g.GdnqError) as e:
        g.gdnq_rope_table(desc, g.RopeFreqs(**kw))
    assert e.value.code == code and msg in str(e.value)


def test_table_null(g):
    d = g.RopeDesc(d=64).c()
    assert g.lib.gdnq_rope_table(d, None, BASE) == 1 and g.lib.gdnq_rope_table(None, None, BASE) == 1
    from recurrent_state_quantization_amd.attn import _RopeFreqs
    assert g.lib.gdnq_rope_table(d, _RopeFreqs(0, 1e4, 1, 0, 0, 0, None), None) == 1


# --------------------------------------------------------------- refusals
def _bufs(names, over):
    return {**{n: BASE + i * (1 << 36) for i, n in enumerate(names)}, **over}


def _err(g, rc):
    return rc, g.lib.gdnq_last_error().decode()


def _rope(g, desc=None, rows=4, H=3, ldx=0, ldy=0, **over):
    d = g.RopeDesc(**{"d": 64, **(desc or {})}).c()
    b = _bufs(["table", "x", "pos", "y"], over)
    return _err(g, g.lib.gdnq_rope(d, b["table"], b["x"], ldx, H, b["pos"], b["y"], ldy, rows, 0))


@pytest.mark.parametrize("kw,code,msg", [
    (dict(desc=dict(d=5)), 2, "d must"),
    (dict(H=0), 1, "H must"),
    (dict(rows=-1), 1, "rows must"),
    (dict(table=None), 1, "table is NULL"),
    (dict(pos=None), 1, "pos is NULL"),
    (dict(x=None), 1, "x is NULL"),
    (dict(y=None), 1, "y is NULL"),
    (dict(pos=BASE + 4), 1, "16-byte"),
    (dict(x=BASE + (1 << 36) + 1), 1, "element size"),
    (dict(ldx=191), 1, "rows of x"),
    (dict(ldy=-5), 1, "rows of y"),
    (dict(y=BASE + (1 << 36) + 2), 1, "y overlaps x"),
    (dict(y=BASE + (1 << 36), ldy=200), 1, "another distance"),
    (dict(y=BASE), 1, "y overlaps table"),
    (dict(desc=dict(d=2), H=2 ** 20, rows=2 ** 11), 1, "too large"),
])
def test_rope_refusals(g, kw, code, msg):
    rc, m = _rope(g, **kw)
    assert rc == code and msg in m, (rc, m)


KV = ["kvk", "kvv", "acc", "kvpos", "kvtable", "lens"]


def _cache(b, kv):
    from recurrent_state_quantization_amd.attn import _Kv
    c = _Kv(*[b[k] for k in KV], 40, 8, 12, 0, 0, 0)
    for k, v in (kv or {}).items():
        setattr(c, k, v)
    return c


def _append(g, desc=None, rope=None, kv=None, n=4, T=64, ld=(0, 0, 0, 0), with_rope=True, no_kv=False, **over):
    d = g.AttnDesc(**{"H": 6, "hk": 2, "d": 64, "page": 16, **(desc or {})}).c()
    r = g.RopeDesc(**{"d": 64, **(rope or {})}).c()
    b = _bufs(["table", "q", "q_out", "k", "v", "pos", "slots", "cu"] + KV, over)
    return _err(g, g.lib.gdnq_kv_append(d, r if with_rope else None, b["table"], None if no_kv else _cache(b, kv),
                                        b["q"], ld[0], b["q_out"], ld[1], b["k"], ld[2], b["v"], ld[3], b["pos"],
                                        b["slots"], b["cu"], n, T, 0))


def _step(g, desc=None, kv=None, n=4, ldq=0, ldo=0, size=1 << 40, no_kv=False, **over):
    d = g.AttnDesc(**{"H": 6, "hk": 2, "d": 64, "page": 16, **(desc or {})}).c()
    b = _bufs(["q", "o", "slots", "ws"] + KV, over)
    return _err(g, g.lib.gdnq_attn_step(d, None if no_kv else _cache(b, kv), b["q"], ldq, b["o"], ldo, b["slots"], n,
                                        b["ws"], size, 0))


def _evict(g, desc=None, kv=None, n=4, budget=96, sink=4, recent=8, size=1 << 40, no_kv=False, **over):
    d = g.AttnDesc(**{"H": 6, "hk": 2, "d": 64, "page": 16, **(desc or {})}).c()
    b = _bufs(["slots", "ws"] + KV, over)
    return _err(g, g.lib.gdnq_kv_evict(d, None if no_kv else _cache(b, kv), budget, sink, recent, b["slots"], n,
                                       b["ws"], size, 0))


CALLS = dict(append=_append, step=_step, evict=_evict)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(desc=dict(H=0)), 1, "H must"),
    (dict(desc=dict(hk=4)), 1, "hk must divide"),
    (dict(desc=dict(hk=-1)), 1, "hk must divide"),
    (dict(desc=dict(d=96)), 2, "d must"),
    (dict(desc=dict(io_dtype=7)), 1, "io_dtype"),
    (dict(desc=dict(page=12)), 2, "page must"),
    (dict(desc=dict(page=4)), 2, "page must"),
    (dict(desc=dict(page=131072)), 2, "page must"),
    (dict(desc=dict(window=-1)), 1, "window"),
    (dict(desc=dict(scale=-1.0)), 1, "scale"),
    (dict(desc=dict(scale=float("inf"))), 1, "scale"),
    (dict(desc=dict(scale=float("nan"))), 1, "scale"),
    (dict(desc=dict(acc_decay=1.5)), 1, "acc_decay"),
    (dict(desc=dict(acc_decay=float("nan"))), 1, "acc_decay"),
    (dict(no_kv=True), 1, "kv is NULL"),
    (dict(kv=dict(n_pages=0)), 1, "n_pages"),
    (dict(kv=dict(n_slots=0)), 1, "n_slots"),
    (dict(kv=dict(max_pages=0)), 1, "max_pages"),
    (dict(kv=dict(max_pages=2 ** 26 + 1)), 2, "2^30 rows"),
    (dict(kv=dict(ldr=64)), 1, "rows of a page overlap"),
    (dict(kv=dict(ldp=4096, ldh=1024)), 1, "rows of a page overlap"),
    (dict(kv=dict(ldp=2048, ldh=960, ldr=64)), 1, "rows of a page overlap"),
    (dict(kv=dict(ldp=2048, ldh=64, ldr=120)), 1, "rows of a page overlap"),
    (dict(kv=dict(ldp=2048, ldh=1025, ldr=64)), 1, "16 bytes"),
    (dict(kv=dict(ldp=1984, ldh=1024, ldr=64)), 1, "pages overlap"),
    (dict(kv=dict(ldp=-2048, ldh=1024, ldr=64)), 1, "0..2^48"),
    (dict(kv=dict(ldp=2 ** 47, ldh=2 ** 41, ldr=2 ** 41)), 1, "larger than any page"),
    (dict(kv=dict(ldp=2 ** 45, ldh=1024, ldr=64), desc=dict(io_dtype=0)), 1, ""),
    (dict(kv=dict(ldp=2 ** 47, ldh=1024, ldr=64, n_pages=2 ** 31 - 1)), 1, "larger than any memory"),
    (dict(n=-1), 1, "must be >= 0"),
    (dict(slots=None, n=9), 1, ""),
    (dict(kvk=None), 1, "kv.k is NULL"),
    (dict(kvv=None), 1, "kv.v is NULL"),
    (dict(kvtable=None), 1, "kv.table is NULL"),
    (dict(lens=None), 1, "kv.lens is NULL"),
    (dict(kvk=BASE + (20 << 36) + 8), 1, "kv.k is not 16-byte"),
    (dict(slots=BASE + (21 << 36) + 4), 1, "slots is not 16-byte"),
])
@pytest.mark.parametrize("call", ["append", "step", "evict"])
def test_cache_refusals(g, call, kw, code, msg):
    if kw == dict(kv=dict(ldp=2 ** 45, ldh=1024, ldr=64), desc=dict(io_dtype=0)):
        kw = dict(kw, kvv=BASE + (22 << 36))   # k's pages reach over the other buffers
    rc, m = CALLS[call](g, **kw)
    assert rc == code and msg in m and m, (rc, m)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(rope=dict(d=128)), 1, "rope is for"),
    (dict(rope=dict(io_dtype=0)), 1, "rope is for"),
    (dict(rope=dict(rot=3)), 1, "rot must"),
    (dict(T=-1), 1, "T must"),
    (dict(cu=None, n=4, T=5), 1, "cu_seqlens is NULL"),
    (dict(table=None), 1, "table is NULL"),
    (dict(k=None), 1, "k is NULL"),
    (dict(v=None), 1, "v is NULL"),
    (dict(q=None), 1, "q and q_out"),
    (dict(q_out=None), 1, "q and q_out"),
    (dict(ld=(383, 0, 0, 0)), 1, "rows of q"),
    (dict(ld=(0, 383, 0, 0)), 1, "rows of q_out"),
    (dict(ld=(0, 0, 127, 0)), 1, "rows of k"),
    (dict(ld=(0, 0, 0, 127)), 1, "rows of v"),
    (dict(q_out=BASE + (1 << 36), ld=(400, 390, 0, 0)), 1, "another distance"),
    (dict(q_out=BASE + (3 << 36)), 1, "k overlaps q_out"),
    # columns of the same rows: the second's run into the first's, by one element, and round the row's end
    (dict(q_out=BASE + (3 << 36) - 766, ld=(0, 700, 700, 0)), 1, "k overlaps q_out"),
    (dict(q_out=BASE + (4 << 36) + 254, ld=(0, 700, 0, 700)), 1, "v overlaps q_out"),
    (dict(q_out=BASE + (3 << 36) + 512, ld=(0, 500, 500, 0)), 1, "k overlaps q_out"),
    (dict(q_out=BASE + (3 << 36) + 256, ld=(0, 700, 640, 0)), 1, "k overlaps q_out"),
    (dict(kvk=BASE + (3 << 36)), 1, "overlaps"),
    (dict(kvv=BASE + (8 << 36)), 1, "kv.v overlaps kv.k"),
    (dict(kvpos=BASE + (10 << 36) + 64), 1, "kv.pos overlaps kv.acc"),
    (dict(lens=BASE + (8 << 36)), 1, "kv.lens overlaps kv.k"),
    (dict(n=2 ** 31 - 1, T=2 ** 31 - 1), 1, ""),
])
def test_append_refusals(g, kw, code, msg):
    rc, m = _append(g, **kw)
    assert rc == code and msg in m, (rc, m)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(q=None), 1, "q is NULL"),
    (dict(o=None), 1, "o is NULL"),
    (dict(ldq=383), 1, "rows of q"),
    (dict(ldo=1), 1, "rows of o"),
    (dict(o=BASE), 1, "o overlaps q"),
    (dict(o=BASE + (4 << 36)), 1, "o overlaps kv.k"),
    (dict(acc=BASE + (4 << 36)), 1, "kv.acc overlaps kv.k"),
    (dict(slots=None, n=9), 1, "slots is NULL"),
    (dict(desc=dict(H=2 ** 27, hk=1), n=16, kv=dict(n_slots=16)), 1, ""),
])
def test_step_refusals(g, kw, code, msg):
    rc, m = _step(g, **kw)
    assert rc == code and msg in m, (rc, m)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(budget=0), 1, "budget must"),
    (dict(sink=-1), 1, "sink and recent"),
    (dict(recent=-1), 1, "sink and recent"),
    (dict(sink=89), 1, "sink and recent"),
    (dict(acc=None), 1, "kv.acc is NULL"),
    (dict(kvpos=None), 1, "kv.pos is NULL"),
    (dict(kvv=BASE + (2 << 36)), 1, "kv.v overlaps kv.k"),
    (dict(size=0), 1, "too small"),
    (dict(ws=None), 1, "workspace is NULL"),
    (dict(ws=BASE + (2 << 36)), 1, "workspace overlaps"),
])
def test_evict_refusals(g, kw, code, msg):
    rc, m = _evict(g, **kw)
    assert rc == code and msg in m, (rc, m)


def test_workspaces(g):
    """Workspaces never shrink with more entries, and too small a one is refused."""
    from recurrent_state_quantization_amd import attn
    for acc in (None, BASE + (6 << 36)):
        b = _bufs(KV, dict(acc=acc))
        for d in (g.AttnDesc(H=6, hk=2, d=64, page=16), g.AttnDesc(H=64, hk=1, d=256, page=8, io_dtype=0)):
            for width in (1, 3, 12, 1000, 2 ** 17):
                kv, last, laste = _cache(b, dict(max_pages=width)), 0, 0
                for n in (0, 1, 2, 3, 7, 8, 100, 513, 4096, 100000):
                    nb = g.gdnq_attn_workspace(d, kv, n)
                    ne = g.gdnq_kv_evict_workspace(d, kv, 64, n)
                    assert nb >= last and ne >= laste and (n or nb == ne == 0)
                    last, laste = nb, ne
    b = _bufs(KV, {})
    nb = g.gdnq_attn_workspace(g.AttnDesc(H=6, hk=2, d=64, page=16), _cache(b, None), 4)
    if nb:
        assert "too small" in _step(g, size=nb - 1)[1]
        assert "overlaps" in _step(g, size=nb, ws=BASE)[1]
    out = ctypes.c_size_t()
    d, kv = g.AttnDesc(H=6, hk=2, d=64, page=16).c(), _cache(b, None)
    for call in (lambda n, o: g.lib.gdnq_attn_workspace(d, kv, n, o),
                 lambda n, o: g.lib.gdnq_kv_evict_workspace(d, kv, 64, n, o)):
        assert call(-1, ctypes.byref(out)) == 1 and call(4, None) == 1
    assert g.lib.gdnq_kv_evict_workspace(d, kv, 0, 4, ctypes.byref(out)) == 1
    assert isinstance(kv, attn._Kv)


@pytest.mark.parametrize("desc,kv,msg", [
    (dict(page=65536), dict(ldp=2 ** 48, ldh=64, ldr=2 ** 48, max_pages=1), "pages overlap"),
    (dict(page=32768), dict(ldp=2 ** 48, ldh=2 ** 39, ldr=2 ** 48, max_pages=1), "pages overlap"),
    (dict(page=65536), dict(ldp=2 ** 48, ldh=2 ** 39, ldr=2 ** 48 - 128, max_pages=1), "pages overlap"),
    (dict(H=2 ** 30, hk=2 ** 30), dict(ldp=2 ** 48, ldh=2 ** 40, ldr=64), "pages overlap"),
    (dict(H=2 ** 30, hk=2 ** 30), dict(ldp=2 ** 48, ldh=2 ** 34, ldr=2 ** 48), "rows of a page overlap"),
    (dict(H=2 ** 31 - 1, hk=2 ** 31 - 1, page=8), dict(ldp=2 ** 48, ldh=2 ** 33, ldr=2 ** 39), "rows of a page overlap"),
])
def test_far_distances(g, desc, kv, msg):
    """Distances whose products with the sizes leave 64 bits are refused by what they are."""
    d = g.AttnDesc(**{**dict(H=6, hk=2, d=64, page=16), **desc}).c()
    c, out = _cache(_bufs(KV, {}), kv), ctypes.c_size_t()
    for rc in (g.lib.gdnq_attn_workspace(d, c, 1, ctypes.byref(out)),
               g.lib.gdnq_kv_evict_workspace(d, c, 64, 1, ctypes.byref(out))):
        rc, m = _err(g, rc)
        assert rc == 1 and msg in m, (rc, m)


@pytest.mark.parametrize("io,H,hk,d,n,rope", [
    (0, 2 ** 26, 1, 256, 1, dict(d=256, io_dtype=0)),             # 2^31 pieces of queries
    (0, 2 ** 27, 1, 256, 1, dict(d=256, io_dtype=0)),             # 2^32
    (1, 2 ** 25, 2 ** 25, 256, 3, dict(d=256, rot=2)),
    (1, 2 ** 23, 2 ** 23, 256, 2000, dict(d=256, rot=14)),        # four rows to a workgroup
    (0, 2 ** 30 - 2, 2 ** 30 - 2, 64, 1, None),
])
def test_append_refuses_rows_beyond_its_numbers(g, io, H, hk, d, n, rope):
    """Rows of more pieces than a workgroup's 31 bits number (hundreds of GB a row)."""
    far = {k: i << 56 for i, k in enumerate(["q", "q_out", "k", "v", "kvk", "kvv", "acc", "kvpos"], 2)}
    rc, m = _append(g, desc=dict(H=H, hk=hk, d=d, io_dtype=io, page=8), rope=rope, with_rope=rope is not None, n=n, T=n,
                    kv=dict(n_pages=1, max_pages=1, n_slots=2000), **far)
    assert rc == 1 and "too many" in m, (rc, m)


def test_append_takes_wide_rows(g):
    """Past the argument checks, to the launch: rows of 2^28 values are within the numbers."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checks only")
    far = {k: i << 56 for i, k in enumerate(["q", "q_out", "k", "v", "kvk", "kvv", "acc", "kvpos"], 2)}
    rc, m = _append(g, desc=dict(H=2 ** 20, hk=2 ** 10, d=256, page=8), rope=dict(d=256), n=2000, T=2000,
                    kv=dict(n_pages=1, max_pages=1, n_slots=2000), **far)
    assert rc == 3, (rc, m)


def test_workspaces_beyond_any_memory(g):
    """Sizes that 64 bits do not count are refused, by the calls too; none is answered with a small one."""
    out = ctypes.c_size_t()

    def sizes(desc, kv, n, budget=64):
        d = g.AttnDesc(**{**dict(H=6, hk=2, d=64, page=16), **desc}).c()
        c = _cache(_bufs(KV, {}), kv)
        return (_err(g, g.lib.gdnq_attn_workspace(d, c, n, ctypes.byref(out))), out.value,
                _err(g, g.lib.gdnq_kv_evict_workspace(d, c, budget, n, ctypes.byref(out))), out.value)

    # 2^31 pages of 2^16 rows, 2^21 heads over one: the scores' bytes are a multiple of 2^64 and a little
    for desc, pages in ((dict(H=2 ** 20, hk=1, page=65536), 2 ** 31 - 1), (dict(H=2 ** 21, hk=1, page=65536), 2 ** 30),
                        (dict(H=2 ** 31 - 1, hk=1), 2 ** 31 - 1)):
        grid = desc["H"] <= 0x7ffffff0   # heads that a grid holds (the first refusal, with sums or without)
        (rc, m), *_ = sizes(desc, dict(n_pages=pages, max_pages=1), 1)
        assert rc == 1 and ("larger than any memory" if grid else "n*H") in m, (rc, m)
        assert sizes(desc, dict(n_pages=pages, max_pages=1, acc=None), 1)[0][0] == (0 if grid else 1)
    kv = dict(n_pages=2 ** 30, max_pages=1)
    rc, m = _step(g, desc=dict(H=2 ** 21, hk=1, page=65536), kv=kv, n=1, kvk=1 << 60, kvv=1 << 61, acc=1 << 59)
    assert rc == 1 and "larger than any memory" in m, (rc, m)
    # entries and heads that no grid holds
    (rc, m), _, (rc2, m2), _ = sizes(dict(H=2 ** 16, hk=2 ** 16), {}, 2 ** 15)
    assert rc == 1 and "n*H" in m and rc2 == 1 and "n*hk" in m2
    # the largest that one does
    for desc, n in ((dict(H=2 ** 26, hk=2 ** 26), 1), (dict(H=1, hk=1, d=256), 2 ** 27 - 1)):
        (rc, m), a, (rc2, m2), b = sizes(desc, dict(max_pages=2 ** 14), n, 2 ** 17)
        assert rc == 0 and rc2 == 0 and n * desc["H"] * 8 <= a < 2 ** 60 and n * desc["H"] * 2 ** 20 <= b < 2 ** 60


def test_append_takes_columns_of_the_same_rows(g):
    """q turned in place beside k and v: past the argument checks, to the launch
    (which fails here, without a GPU, or would fault on these addresses with one: not run there)."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checks only")
    at = BASE + (1 << 36)
    for q, k, v, ld in ((0, 768, 1024, 640), (512, 0, 256, 640), (128, 1792 + 128, 896, 1024)):
        rc, m = _append(g, q=at + q, q_out=at + q, k=at + k, v=at + v, ld=(ld, ld, ld, ld))
        assert rc == 3, (rc, m)


# keys and values in one pool of 40 pages of 16 rows, 2 heads, 64 bf16 values: ldp, ldh, ldr, and where v is, in
# elements behind k
POOLS = {"pages": (4096, 1024, 64, 2048), "heads": (4096, 2048, 64, 1024), "rows": (4096, 2048, 128, 64),
         "pages of rows of heads": (4096, 64, 128, 2048), "rows of heads": (4096, 64, 256, 128),
         "heads of rows": (4096, 128, 256, 64), "v first": (4096, 1024, 64, -2048),
         "gaps": (8192, 64, 256, 4096 + 128), "pages behind": (4096, 1024, 64, 5 * 4096 + 2048)}


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("call", ["append", "evict"])
def test_one_pool_of_keys_and_values(g, call, pool):
    """Past the argument checks, to the launch (which fails here, without a GPU)."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checks only")
    ldp, ldh, ldr, by = POOLS[pool]
    at = BASE + (20 << 36)
    rc, m = CALLS[call](g, kvk=at, kvv=at + 2 * by, kv=dict(ldp=ldp, ldh=ldh, ldr=ldr))
    assert rc == 3, (rc, m)


def _meet(ldp, ldh, ldr, by, d=64, n_pages=40, hk=2, page=16):
    rows = sorted(p * ldp + h * ldh + r * ldr for p in range(n_pages) for h in range(hk) for r in range(page))
    both = sorted([(x, 0) for x in rows] + [(x + by, 1) for x in rows])
    return any(b[0] - a[0] < d for a, b in zip(both, both[1:]))


@pytest.mark.parametrize("ld", sorted({p[:3] for p in POOLS.values()}))
def test_pools_whose_rows_meet(g, ld):
    """Every distance of v from k, in pieces of 16 bytes: refused where a row of the one
    meets a row of the other (found row by row), and only there."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checks only")
    at, seen = BASE + (20 << 36), set()
    kv = dict(ldp=ld[0], ldh=ld[1], ldr=ld[2])
    for by in [*range(-400, 401, 8), *range(ld[0] - 136, ld[0] + 137, 8), *range(ld[0] // 2 - 72, ld[0] // 2 + 73, 8),
               *range(39 * ld[0] - 72, 40 * ld[0], 1016), *range(-38 * ld[0] - 640, -37 * ld[0], 328)]:
        rc, m = _evict(g, kvk=at, kvv=at + 2 * by, kv=kv)
        meet = _meet(*ld, by)
        assert (rc == 1 and "kv.v overlaps kv.k" in m) if meet else rc == 3, (by, rc, m)
        seen.add(meet)
    assert seen == {False, True}


@pytest.mark.parametrize("kw,msg", [
    (dict(acc=BASE + (20 << 36) + 4096), "kv.acc overlaps kv.k"),
    (dict(acc=BASE + (20 << 36) + 80 * 4096 - 16), "kv.acc overlaps kv.v"),
    (dict(slots=BASE + (20 << 36) + 80 * 4096 - 16), "kv.v overlaps slots"),
    (dict(lens=BASE + (20 << 36) + 80 * 4096 - 16), "kv.lens overlaps kv.v"),
])
def test_one_pool_beside_others(g, kw, msg):
    """A pool of both overlaps no other buffer (the last values lie behind the last keys)."""
    at = BASE + (20 << 36)
    for call in ("append", "evict"):
        rc, m = CALLS[call](g, kvk=at, kvv=at + 4096, kv=dict(ldp=4096, ldh=1024, ldr=64), **kw)
        assert rc == 1 and msg in m, (rc, m)


def test_no_ops(g):
    """Calls of nothing touch no pointer."""
    assert _rope(g, rows=0, x=None, y=None)[0] == 0
    assert _append(g, n=0, k=None)[0] == 0 and _append(g, T=0, k=None)[0] == 0
    assert _step(g, n=0, q=None)[0] == 0
    assert _evict(g, n=0, acc=None)[0] == 0
    assert _evict(g, budget=12 * 16, size=0, ws=None)[0] == 0   # no slot holds more


# ------------------------------------------------------------ the binding
def test_binding_refuses_tensors(g):
    """Tensors off the GPU, of another type or shape never reach the library."""
    torch = pytest.importorskip("torch")
    x, pos = torch.zeros(4, 3 * 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    table = g.gdnq_rope_table(g.RopeDesc(d=64), g.RopeFreqs())
    with pytest.raises(g.GdnqError, match="not on a GPU"):
        g.gdnq_rope(g.RopeDesc(d=64), table, x, pos, x, 4, 3, 0)
    with pytest.raises(g.GdnqError, match="int64"):
        g.gdnq_rope(g.RopeDesc(d=64), table.float(), BASE, BASE, BASE, 4, 3, 0)
    k = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)
    kv = g.Kv(k, k, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(g.GdnqError, match="not on a GPU"):
        kv.c(g.AttnDesc(H=4, hk=2, d=64, page=16))
    d = g.AttnDesc(H=6, hk=2, d=64, page=16)
    b = _cache(_bufs(KV, {}), None)
    with pytest.raises(g.GdnqError, match="not on a GPU"):
        g.gdnq_attn_step(d, b, torch.zeros(4, 384, dtype=torch.bfloat16), BASE, None, 4, BASE, 0)
    with pytest.raises(g.GdnqError, match="not on a GPU"):
        k = torch.zeros(4, 128, dtype=torch.bfloat16)
        g.gdnq_kv_append(d, None, None, b, None, None, k, BASE, None, None, None, 4, 4, 0)
    with pytest.raises(g.GdnqError, match="not on a GPU"):
        g.gdnq_kv_evict(d, b, 64, 0, 0, torch.zeros(4, dtype=torch.int32), 4, BASE, 0)
