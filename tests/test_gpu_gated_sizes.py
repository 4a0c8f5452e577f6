"""Every pair of head sizes of the gated entry points, in both types, at lengths on
either side of where another kernel takes over (tests/_gated.py: the 64-bit form and
the tolerances)."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _gated as G
from tests import _gated_regimes as R
from tests.test_gpu_gated import GRADS, dev, grads_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DIMS = [16, 32, 64, 128]


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
@pytest.mark.parametrize("dv", DIMS)
@pytest.mark.parametrize("dk", DIMS)
def test_forward_and_backward(dk, dv, dt):
    for B, L, H, Hk, rule in ((1, 9, 2, 1, "exact"), (1, 33, 3, 3, "euler"), (2, 70, 4, 2, "exact"), (1, 193, 8, 4, "euler")):
        x = R.slow(B, L, H, Hk, dk, dv, dt, seed=L + dk + dv)
        gen = torch.Generator().manual_seed(L)
        do, dsf = torch.randn(B, L, H, dv, generator=gen).to(dt), torch.randn(B, H, dk, dv, generator=gen)
        a = dev(x)
        args = [a[n] for n in G.NAMES]
        o, S = efla.efla_gated_chunk_fwd(*args, a["s0"], rule=rule)
        wo, wS = G.forward_ref(*G.wide(x), x["s0"].double(), rule)
        assert G.rel(o, wo) <= G.tol_o(dt, L, dk) and G.rel(S, wS) <= G.tol_s(dt, L, dk), (L, "forward")
        got = efla.efla_gated_chunk_bwd(*args, do.cuda(), a["s0"], dsf.cuda(), rule=rule)
        for n, g, w in zip(GRADS, got, grads_ref(x, do, dsf, rule)):
            assert G.rel(g, w) <= G.tol_grad(dt, L, dk), (L, n)


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
@pytest.mark.parametrize("dv", DIMS)
@pytest.mark.parametrize("dk", DIMS)
def test_step(dk, dv, dt):
    """A few rows, and as many as make the widest value blocks."""
    for N, H, Hk in ((3, 6, 2), (300, 8, 8)):
        x = R.slow(N, 1, H, Hk, dk, dv, dt, seed=N + dk + dv)
        a = dev(x)
        st = a["s0"].clone()
        o = efla.efla_gated_step(*(a[n][:, 0].contiguous() for n in G.NAMES), st)
        wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
        assert G.rel(o, wo[:, 0]) <= G.tol32(1, dk) + (0 if dt == F32 else 2.0 ** -8)
        assert G.rel(st, wS) <= G.tol32(1, dk)


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
@pytest.mark.parametrize("dk,dv", [(16, 128), (32, 32), (64, 32), (128, 32), (64, 16), (128, 128)])
def test_packed(dk, dv, dt):
    lens, H, Hk = [1, 260, 0, 17, 64, 65], 3, 3
    T = sum(lens)
    x = R.slow(len(lens), 0, H, Hk, dk, dv, dt, seed=T + dk + dv, lead=(T,))
    a = dev(x)
    p = efla.efla_pack_plan(torch.tensor(lens, dtype=torch.int32).cuda(), T)
    o, S = efla.efla_gated_chunk_fwd_varlen(*(a[n] for n in G.NAMES), p.cu_seqlens, a["s0"])
    at = 0
    for i, n in enumerate(lens):
        wo, wS = G.forward_ref(*(t[None, at:at + n] for t in G.wide(x)), x["s0"][i:i + 1].double())
        assert n == 0 or G.rel(o[at:at + n], wo[0]) <= G.tol_o(dt, n, dk), (i, "o")
        assert G.rel(S[i], wS[0]) <= G.tol_s(dt, n, dk), (i, "S")
        at += n
