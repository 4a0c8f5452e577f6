"""The inputs of tests/test_gpu_gated_regimes.py, on the CPU: with the carry over a
full chunk left out, every output and every gradient leaves its tolerance."""
import pytest
import torch

from tests import _gated as G
from tests import _gated_regimes as R

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rule", ["exact", "euler"])
@pytest.mark.parametrize("L", [64, 200, 321])
def test_chunk_algebra_of_slow_heads_is_the_recurrence(L, rule):
    x = R.slow(2, L, 4, 2, 16, 8, torch.float64, seed=L)
    a, s0 = G.wide(x), x["s0"].double()
    o, S = G.forward_ref(*a, s0, rule)
    o2, S2 = R.chunked(*a, s0, rule)
    assert G.rel(o2, o) < 1e-12 and G.rel(S2, S) < 1e-12


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("L", [200, 321])
def test_a_lost_carry_leaves_every_tolerance(L, d, dt):
    x = R.slow(1, L, 4, 2, d, d, dt, seed=L + d)
    gen = torch.Generator().manual_seed(1)
    do, dsf = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((1, L, 4, d), (1, 4, d, d)))

    def run(carry):
        leaves = [t.requires_grad_() for t in (*G.wide(x), x["s0"].double())]
        o, S = R.chunked(*leaves, "exact", carry)
        return o, S, torch.autograd.grad((o * do).sum() + (S * dsf).sum(), leaves)

    (o, S, gr), (o2, S2, gr2) = run(True), run(False)
    assert G.rel(o2, o) > 2 * G.tol_o(dt, L, d) and G.rel(S2, S) > 2 * G.tol_s(dt, L, d)
    for name, a, b in zip(("dq", "dk", "dv", "dbeta", "dg", "ds0"), gr2, gr):
        assert G.rel(a, b) > 2 * G.tol_grad(dt, L, d), name
