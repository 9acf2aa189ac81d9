"""Calls of more threads than one dimension of a grid holds (2^32): narrow
rows and small groups reach that at a few GB."""
import pytest

from tests._gpu import lib, say, torch_cuda

pytestmark = pytest.mark.gpu


def test_norms_of_many_rows():
    """One value a row: y = x / sqrt(x^2 + eps)."""
    torch = torch_cuda()
    g = lib()
    rows = (1 << 28) + 77
    say("norms of many rows", rows)
    x = torch.full((rows, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    x[-1] = -3.0
    x[1 << 28] = 5.0
    w = torch.ones(1, device="cuda")
    d = g.NormDesc(D=1)
    y, ro = torch.zeros_like(x), torch.zeros_like(x)
    want = torch.sign(x.float()).bfloat16()
    g.gdnq_norm_gated(d, x, None, w, y, rows)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    g.gdnq_norm_residual(d, x, None, 1.0, x.clone(), ro, w, y, rows)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(ro, x + x)


def test_norms_of_many_small_groups():
    torch = torch_cuda()
    g = lib()
    rows, D, group = (1 << 19) + 3, 4096, 8
    say("norms of many groups", rows, D, group)
    x = torch.full((rows, D), 2.0, dtype=torch.bfloat16, device="cuda")
    x[-1, -8:] = -3.0
    y = torch.zeros_like(x)
    g.gdnq_norm_gated(g.NormDesc(D=D, group=group, flags=g.NORM_GROUP_WEIGHT), x, None,
                      torch.ones(group, device="cuda"), y, rows)
    torch.cuda.synchronize()
    assert bool((y[:-1] == 1).all()) and bool((y[-1, -8:] == -1).all()) and bool((y[-1, :-8] == 1).all())


def test_convolution_of_many_rows():
    torch = torch_cuda()
    g = lib()
    T = (1 << 30) + 33
    say("convolution of many rows", T)
    x = torch.ones(T, 1, dtype=torch.bfloat16, device="cuda")
    x[-1], x[-40] = 3.0, 5.0
    y, st = torch.zeros_like(x), torch.zeros(2, 1, 1, dtype=torch.bfloat16, device="cuda")
    w = torch.tensor([[1.0], [2.0]], device="cuda")
    cu = torch.tensor([0, 5, T], dtype=torch.int32, device="cuda")
    g.gdnq_conv_prefill(g.ConvDesc(C=1, width=2, flags=0), x, w, None, st, 2, None, None, cu, 2, T, y)
    torch.cuda.synchronize()
    want = 2 * x
    want[1:] += x[:-1]
    want[5] = 2 * x[5]
    assert torch.equal(y, want) and st.flatten().tolist() == [1.0, 3.0]


def test_convolution_tokens_of_many_entries():
    torch = torch_cuda()
    g = lib()
    n = (1 << 26) + 9
    say("convolution of many entries", n)
    x = torch.ones(n, 1, dtype=torch.bfloat16, device="cuda")
    x[-1] = 3.0
    y = torch.zeros_like(x)
    st = torch.full((n, 1, 1), 4.0, dtype=torch.bfloat16, device="cuda")
    w = torch.tensor([[1.0], [2.0]], device="cuda")
    g.gdnq_conv_step(g.ConvDesc(C=1, width=2, flags=0), x, w, None, st, n, None, n, y)
    torch.cuda.synchronize()
    assert torch.equal(y, 2 * x + 4) and torch.equal(st.view(n, 1), x)


def test_scan_tokens_of_many_entries():
    """All but a few entries are skipped, so few states are needed."""
    torch = torch_cuda()
    g = lib()
    n, d = (1 << 24) + 5, 64
    say("scan of many entries", n)
    keep = [0, 1 << 23, (1 << 24) - 1, 1 << 24, n - 1]
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[keep] = torch.arange(5, dtype=torch.int32, device="cuda")
    one = lambda w: torch.ones(n, w, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, B, dt = one(d), one(d), one(1)
    y = torch.zeros_like(x)
    S = torch.zeros(5, 1, d, d, device="cuda")
    g.gdnq_ssm_step(g.SsmDesc(H=1, dk=d, dv=d, flags=0), x, B, B, dt, torch.zeros(1, device="cuda"), None, None, y, S, 5,
                    slots, n)
    torch.cuda.synchronize()
    assert bool((y[keep] == d).all()) and bool((S == 1).all())
    y[keep] = 0
    assert not bool(y.any())
