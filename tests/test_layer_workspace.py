"""The scan's workspace (gdnq_ssm_workspace) over sequences and token rows:
what a call needs, every call of fewer sequences and rows needs no more."""
import random

import pytest


@pytest.fixture(scope="module")
def g():
    import recurrent_state_quantization_amd as g
    return g


@pytest.mark.parametrize("H,dk,dv,hk", [(24, 128, 64, 1), (64, 128, 64, 1), (32, 128, 128, 8), (80, 128, 64, 1),
                                        (1, 64, 64, 1), (93, 128, 128, 1), (48, 64, 64, 48), (300, 64, 128, 300),
                                        (2000, 64, 64, 2000)])
def test_workspace_never_shrinks(g, H, dk, dv, hk):
    d = g.SsmDesc(H=H, dk=dk, dv=dv, hk=hk)
    ws = lambda n, T: g.gdnq_ssm_workspace(d, n, T)  # noqa: E731
    for n in (1, 2, 9, 300):
        at = [ws(n, T) for T in range(1, 9000, 3)] + [ws(n, T) for T in range(9000, 300000, 997)]
        assert at == sorted(at), (n, next(i for i in range(1, len(at)) if at[i] < at[i - 1]))
    for T in (200, 385, 2048, 5269, 40000):
        at = [ws(n, T) for n in range(1, 600)]
        assert at == sorted(at), T
    r = random.Random(H)
    for _ in range(3000):
        n, T = r.randrange(1, 2000), r.randrange(1, 100000)
        assert ws(r.randrange(1, n + 1), r.randrange(1, T + 1)) <= ws(n, T)


def test_workspace_of_a_long_call_is_as_large_as_its_shares(g):
    """64 heads in blocks of 4 are 16 workgroups a share, so 16 shares fill 256
    compute units: two states and an exponent for each and every head."""
    assert g.gdnq_ssm_workspace(g.SsmDesc(H=64, dk=128, dv=64, hk=1), 1, 16384) == 16 * 64 * (2 * 128 * 64 + 1) * 4


def test_more_workgroups_than_a_grid_holds(g):
    """Sequences of a short call without tokens still take workgroups."""
    from recurrent_state_quantization_amd import layer
    base, far = 1 << 40, 1 << 36
    io = layer._SsmIo(*[base + i * far for i in range(8)], 0, 0, 0, 0, 0)
    d = g.SsmDesc(H=64, dk=64, dv=64, hk=64).c()
    p = [base + i * far for i in range(8, 13)]
    rc = g.lib.gdnq_ssm_prefill(d, io, p[0], 2, p[1], None, p[2], 1 << 19, 384, p[3], 1 << 30, 0)
    assert rc == 1 and "n_seqs*H" in g.lib.gdnq_last_error().decode()
