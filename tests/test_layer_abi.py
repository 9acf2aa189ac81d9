"""The C ABI of include/gdnq_layer.h without a GPU: exports, struct layouts,
and the refusal of every invalid argument on the host.  Device pointers are
fake aligned addresses: a rejected call never dereferences them."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdnq_layer.h")
NAMES = ["gdnq_conv_prefill", "gdnq_conv_step", "gdnq_norm_gated", "gdnq_norm_residual", "gdnq_ssm_prefill",
         "gdnq_ssm_step", "gdnq_ssm_workspace"]
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


@pytest.mark.parametrize("name,mirror", [("gdnq_conv_desc", "_ConvDesc"), ("gdnq_ssm_desc", "_SsmDesc"),
                                         ("gdnq_ssm_io", "_SsmIo"), ("gdnq_norm_desc", "_NormDesc")])
def test_struct_layouts_match_header(g, name, mirror):
    from recurrent_state_quantization_amd import layer
    body = [b for b, n in re.findall(r"typedef struct \{([^}]*)\} (\w+);", _text()) if n == name][0]
    assert re.findall(r"(\w+)(?=\s*[,;])", body) == [f[0] for f in getattr(layer, mirror)._fields_]


def test_flag_values_match_header(g):
    text = open(HEADER).read()
    for k in ("CONV_SILU", "SSM_SOFTPLUS", "NORM_GATE_SIGMOID", "NORM_GATE_FIRST", "NORM_GROUP_WEIGHT", "NORM_RES_F32"):
        assert int(re.search(rf"#define GDNQ_{k} (\d+)u", text).group(1)) == getattr(g, k)


def test_header_is_c(tmp_path):
    f = tmp_path / "t.c"
    f.write_text('#include "gdnq_layer.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER), str(f)],
                   check=True)


class Fake:
    """Disjoint fake buffers by name, replaced by keyword."""

    def __init__(self, names):
        self.p = {n: BASE + i * (1 << 36) for i, n in enumerate(names)}

    def __call__(self, **over):
        return {**self.p, **over}


def _err(g, rc_fn):
    rc = rc_fn()
    return rc, g.lib.gdnq_last_error().decode()


def _conv(g, desc=None, step=False, n=4, T=64, n_slots=8, ldx=0, ldy=0, **over):
    d = g.ConvDesc(**{"C": 64, **(desc or {})}).c()
    b = Fake(["x", "w", "bias", "state", "slots", "cont", "cu", "y"])(**over)
    if step:
        return _err(g, lambda: g.lib.gdnq_conv_step(d, b["x"], ldx, b["w"], b["bias"], b["state"], n_slots, b["slots"],
                                                    n, b["y"], ldy, 0))
    return _err(g, lambda: g.lib.gdnq_conv_prefill(d, b["x"], ldx, b["w"], b["bias"], b["state"], n_slots, b["slots"],
                                                   b["cont"], b["cu"], n, T, b["y"], ldy, 0))


def _ssm(g, desc=None, step=False, n=4, T=64, n_slots=8, ws=None, ld=None, **over):
    from recurrent_state_quantization_amd import layer
    d = g.SsmDesc(**{"H": 4, "hk": 2, **(desc or {})}).c()
    b = Fake(["x", "B", "C", "dt", "y", "A", "D", "dt_bias", "S", "slots", "cont", "cu", "ws"])(**over)
    io = layer._SsmIo(*[b[k] for k in ("x", "B", "C", "dt", "y", "A", "D", "dt_bias")], 0, 0, 0, 0, 0)
    for k, v in (ld or {}).items():
        setattr(io, k, v)
    if step:
        return _err(g, lambda: g.lib.gdnq_ssm_step(d, io, b["S"], n_slots, b["slots"], n, 0))
    size = 1 << 34 if ws is None else ws
    return _err(g, lambda: g.lib.gdnq_ssm_prefill(d, io, b["S"], n_slots, b["slots"], b["cont"], b["cu"], n, T, b["ws"],
                                                  size, 0))


def _gated(g, desc=None, rows=4, ldx=0, ldz=0, ldy=0, **over):
    d = g.NormDesc(**{"D": 256, "group": 64, **(desc or {})}).c()
    b = Fake(["x", "z", "w", "y"])(**over)
    return _err(g, lambda: g.lib.gdnq_norm_gated(d, b["x"], ldx, b["z"], ldz, b["w"], b["y"], ldy, rows, 0))


def _res(g, desc=None, rows=4, scale=1.0, ldx=0, ldr=0, ldro=0, ldy=0, **over):
    d = g.NormDesc(**{"D": 256, **(desc or {})}).c()
    b = Fake(["x", "post_w", "res", "res_out", "w", "y"])(**over)
    return _err(g, lambda: g.lib.gdnq_norm_residual(d, b["x"], ldx, b["post_w"], scale, b["res"], ldr, b["res_out"],
                                                    ldro, b["w"], b["y"], ldy, rows, 0))


@pytest.mark.parametrize("kw,code,msg", [
    (dict(desc=dict(C=0)), 1, "C must"),
    (dict(desc=dict(width=1)), 2, "width"),
    (dict(desc=dict(width=5)), 2, "width"),
    (dict(desc=dict(io_dtype=3)), 1, "io_dtype"),
    (dict(desc=dict(flags=2)), 1, "flag"),
    (dict(n=-1), 1, "must be >= 0"),
    (dict(n_slots=0), 1, "n_slots"),
    (dict(slots=None, n_slots=3), 1, "slots is NULL"),
    (dict(x=None), 1, "x is NULL"),
    (dict(y=None), 1, "y is NULL"),
    (dict(w=None), 1, "w is NULL"),
    (dict(state=None), 1, "state is NULL"),
    (dict(x=BASE + 1), 1, "element size"),
    (dict(w=BASE + (9 << 36) + 4), 1, "16-byte"),
    (dict(ldx=63), 1, "rows of x"),
    (dict(ldy=-1), 1, "rows of y"),
    (dict(y=BASE), 1, "y overlaps x"),
    (dict(state=BASE + 64), 1, "state overlaps x"),
    (dict(y=BASE + (3 << 36) + 128), 1, "y overlaps state"),
    (dict(y=BASE + (4 << 36)), 1, "y overlaps slots"),
    (dict(desc=dict(C=2 ** 31 - 1), n=2 ** 31 - 1, n_slots=2 ** 31 - 1), 1, ""),
])
@pytest.mark.parametrize("step", [False, True])
def test_conv_refusals(g, kw, code, msg, step):
    rc, m = _conv(g, step=step, **kw)
    assert rc == code and msg in m and m, (rc, m)


def test_conv_packed_refusals(g):
    assert _conv(g, T=-1)[0] == 1
    rc, m = _conv(g, cu=None)
    assert rc == 1 and "cu_seqlens is NULL" in m
    rc, m = _conv(g, y=BASE + (6 << 36))
    assert rc == 1 and "y overlaps cu_seqlens" in m


@pytest.mark.parametrize("kw,code,msg", [
    (dict(desc=dict(H=0)), 1, "H must"),
    (dict(desc=dict(dk=96)), 2, "dk and dv"),
    (dict(desc=dict(dv=256)), 2, "dk and dv"),
    (dict(desc=dict(hk=3)), 1, "hk must divide"),
    (dict(desc=dict(hk=-1)), 1, "hk must divide"),
    (dict(desc=dict(io_dtype=9)), 1, "io_dtype"),
    (dict(desc=dict(flags=4)), 1, "flag"),
    (dict(desc=dict(dt_min=-1.0)), 1, "dt_min"),
    (dict(desc=dict(dt_min=0.2, dt_max=0.1)), 1, "dt_min"),
    (dict(n=-2), 1, "must be >= 0"),
    (dict(n_slots=0), 1, "n_slots"),
    (dict(slots=None, n_slots=1), 1, "slots is NULL"),
    (dict(S=None), 1, "S is NULL"),
    (dict(A=None), 1, "A is NULL"),
    (dict(dt=None), 1, "dt is NULL"),
    (dict(ld=dict(ldx=255)), 1, "rows of x"),
    (dict(ld=dict(ldb=255)), 1, "rows of B"),
    (dict(ld=dict(lddt=3)), 1, "rows of dt"),
    (dict(B=BASE + (1 << 36) + 1), 1, "element size"),
    (dict(S=BASE + (8 << 36) + 4), 1, "16-byte"),
    (dict(y=BASE), 1, "y overlaps x"),
    (dict(S=BASE), 1, "S overlaps x"),
    (dict(y=BASE + (8 << 36)), 1, "y overlaps S"),
    (dict(desc=dict(H=2 ** 31 - 1, hk=1), n_slots=2 ** 31 - 1), 1, ""),
])
@pytest.mark.parametrize("step", [False, True])
def test_ssm_refusals(g, kw, code, msg, step):
    rc, m = _ssm(g, step=step, **kw)
    assert rc == code and msg in m and m, (rc, m)


def test_ssm_prompt_refusals(g):
    rc, m = _ssm(g, desc=dict(io_dtype=g.IO_F32))
    assert rc == 2 and "bf16" in m
    assert _ssm(g, T=-1)[0] == 1
    assert "cu_seqlens" in _ssm(g, cu=None)[1]
    big = g.SsmDesc(H=4, hk=1)
    nb = g.gdnq_ssm_workspace(big, 1, 1 << 16)
    if nb:
        rc, m = _ssm(g, desc=dict(hk=1), n=1, T=1 << 16, ws=nb - 1)
        assert rc == 1 and "too small" in m
        rc, m = _ssm(g, desc=dict(hk=1), n=1, T=1 << 16, ws=nb, y=BASE + (12 << 36))
        assert rc == 1 and "overlaps" in m
    out = ctypes.c_size_t()
    assert g.lib.gdnq_ssm_workspace(big.c(), -1, 4, ctypes.byref(out)) == 1
    assert g.lib.gdnq_ssm_workspace(big.c(), 1, 4, None) == 1
    assert g.gdnq_ssm_workspace(big, 0, 100) == 0 and g.gdnq_ssm_workspace(big, 5, 0) == 0


@pytest.mark.parametrize("kw,code,msg", [
    (dict(desc=dict(D=0, group=0)), 1, "D must"),
    (dict(desc=dict(D=32769, group=0)), 2, "32768"),
    (dict(desc=dict(group=100)), 1, "group must divide"),
    (dict(desc=dict(io_dtype=-1)), 1, "io_dtype"),
    (dict(desc=dict(flags=8)), 1, "flag"),
    (dict(desc=dict(eps=0.0)), 1, "eps"),
    (dict(rows=-1), 1, "rows must"),
    (dict(x=None), 1, "x is NULL"),
    (dict(w=None), 1, "w is NULL"),
    (dict(y=None), 1, "y is NULL"),
    (dict(ldz=255), 1, "rows of z"),
    (dict(y=BASE), 1, "y overlaps x"),
    (dict(y=BASE + (1 << 36) + 512), 1, "y overlaps z"),
    (dict(desc=dict(D=32768, group=1), rows=2 ** 31 - 1), 1, ""),
])
def test_gated_refusals(g, kw, code, msg):
    rc, m = _gated(g, **kw)
    assert rc == code and msg in m, (rc, m)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(desc=dict(group=64)), 2, "whole rows"),
    (dict(desc=dict(flags=1)), 1, "flag"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(res=None), 1, "res is NULL"),
    (dict(res_out=None), 1, "res_out is NULL"),
    (dict(w=None), 1, "w is NULL"),
    (dict(res_out=BASE + (2 << 36), ldro=300), 1, "another distance"),
    (dict(res_out=BASE + (2 << 36) + 16), 1, "res_out overlaps res"),
    (dict(res_out=BASE), 1, "res_out overlaps x"),
    (dict(y=BASE + (2 << 36)), 1, "y overlaps res"),
    (dict(y=BASE), 1, "y overlaps x"),
])
def test_residual_refusals(g, kw, code, msg):
    rc, m = _res(g, **kw)
    assert rc == code and msg in m, (rc, m)


def test_empty_calls_return_without_a_launch(g):
    """No rows, sequences or tokens: nothing to do, and no pointer is needed."""
    none = dict.fromkeys(["x", "w", "bias", "state", "slots", "cont", "cu", "y"])
    assert _conv(g, T=0, **none) == (0, "") and _conv(g, n=0, **none) == (0, "")
    assert _conv(g, step=True, n=0, **none) == (0, "")
    none = dict.fromkeys(["x", "B", "C", "dt", "y", "A", "D", "dt_bias", "S", "slots", "cont", "cu", "ws"])
    assert _ssm(g, T=0, **none) == (0, "") and _ssm(g, n=0, **none) == (0, "") and _ssm(g, step=True, n=0, **none) == (0, "")
    assert _gated(g, rows=0, **dict.fromkeys("xzwy")) == (0, "")
    assert _res(g, rows=0, **dict.fromkeys(["x", "post_w", "res", "res_out", "w", "y"])) == (0, "")


def test_null_descriptors(g):
    assert g.lib.gdnq_conv_step(None, 0, 0, 0, 0, 0, 1, 0, 1, 0, 0, 0) == 1
    assert g.lib.gdnq_ssm_step(None, None, 0, 1, 0, 1, 0) == 1
    assert g.lib.gdnq_ssm_step(g.SsmDesc(H=2).c(), None, 0, 1, 0, 1, 0) == 1
    assert "io is NULL" in g.lib.gdnq_last_error().decode()
    assert g.lib.gdnq_norm_gated(None, 0, 0, 0, 0, 0, 0, 0, 1, 0) == 1


def test_binding_refuses_host_tensors_and_other_types(g):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(g.GdnqError, match="not on a GPU"):
        g.gdnq_conv_step(g.ConvDesc(C=64), x, BASE, None, BASE, 4, None, 4, BASE, stream=0)
    from recurrent_state_quantization_amd import layer

    class OnGpu:   # a tensor's face, as the binding sees one on device `index`
        def __init__(self, t, index=0):
            self.t, self.index = t, index

        def get_device(self):
            return self.index

        def __getattr__(self, k):
            return getattr(self.t, k)

    bf = torch.bfloat16
    assert layer._rows(OnGpu(x), 4, 64, bf, 0, "x") == (x.data_ptr(), 64)
    assert layer._rows(OnGpu(x[:, 8:40]), 4, 32, bf, 0, "x")[1] == 64
    assert layer._rows(OnGpu(x.view(4, 2, 32)), 4, 64, bf, 0, "x")[1] == 64
    assert layer._rows(OnGpu(x[:1, :8]), 1, 8, bf, 0, "x")[1] >= 8
    for t, n, w, msg in ((x, 5, 64, "4 rows"), (x, 4, 32, "rows of 32"), (x.float(), 4, 64, "float32"),
                         (x.t(), 4, 4, "consecutive"), (x[:1].expand(4, 64), 4, 64, "overlap"),
                         (x.view(4, 2, 32).transpose(0, 1), 2, 128, "consecutive")):
        with pytest.raises(g.GdnqError, match=msg):
            layer._rows(OnGpu(t), n, w, bf, 0, "x")
    for t, n, msg in ((x[:, ::2], 4, "contiguous"), (x, 257, "values"), (x.float(), 4, "float32")):
        with pytest.raises(g.GdnqError, match=msg):
            layer._flat(OnGpu(t), n, bf, 0, "w")
    for f in (lambda t: layer._flat(t, 4, bf, 0, "w"), lambda t: layer._rows(t, 4, 64, bf, 0, "w")):
        with pytest.raises(g.GdnqError, match="current device"):
            f(OnGpu(x, 1))


@pytest.mark.parametrize("name", ["ldx", "ldb", "ldc", "lddt", "ldy"])
def test_ssm_prompt_rows_far_apart(g, name):
    rc, m = _ssm(g, T=2, ld={name: (1 << 22) + 1})
    assert rc == 2 and "2^22" in m


@pytest.mark.parametrize("H,dk,dv,hk", [(1, 64, 64, 1), (64, 128, 64, 1), (32, 128, 128, 8), (600, 64, 128, 600)])
def test_ssm_workspace_bounds(g, H, dk, dv, hk):
    """None for a call of few tokens; never more than two states and a decay
    for each 64 tokens of all sequences with 192 more each."""
    d = g.SsmDesc(H=H, dk=dk, dv=dv, hk=hk)
    one = H * (2 * dk * dv + 1) * 4
    for n in (1, 3, 1000, 2 ** 20):
        assert g.gdnq_ssm_workspace(d, n, 384) == 0
        for T in (385, 5000, 2 ** 20, 2 ** 31 - 1):
            nb = g.gdnq_ssm_workspace(d, n, T)
            assert nb % one == 0 and 0 <= nb // one <= (T + 192 * n) // 64 + 1 and nb // one <= 6 * 256
