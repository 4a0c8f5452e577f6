"""dg in float32 on the GPU: the sum that is rounded where dg is in the inputs' type."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _gated as G
from tests import _gated_regimes as R
from tests.test_gpu_gated import dev, grads_ref, ids

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("p", [(1, 200, 4, 2, 128, 128, BF), (2, 150, 4, 4, 64, 64, BF), (1, 16, 4, 2, 64, 64, BF),
                               (2, 90, 2, 1, 32, 32, BF), (1, 100, 2, 2, 64, 64, F32)], ids=ids)
def test_float32_gate_gradient(p):
    B, L, H, Hk, dk, dv, dt = p
    x = R.slow(B, L, H, Hk, dk, dv, dt, seed=L)
    gen = torch.Generator().manual_seed(3)
    do, dsf = torch.randn(B, L, H, dv, generator=gen).to(dt), torch.randn(B, H, dk, dv, generator=gen)
    a = dev(x)
    args = (*(a[n] for n in G.NAMES), do.cuda(), a["s0"], dsf.cuda())
    one, two = efla.efla_gated_chunk_bwd(*args), efla.efla_gated_chunk_bwd(*args, dg_dtype=F32)
    assert two[4].dtype == F32 and one[4].dtype == dt and two[4].shape == one[4].shape
    assert torch.equal(two[4].to(dt), one[4])
    for i in (0, 1, 2, 3, 5):
        assert torch.equal(one[i], two[i])
    err = G.rel(two[4], grads_ref(x, do, dsf, "exact")[4])
    # float32 passes (float32 inputs, d 32, at most 16 tokens): float32 throughout; else all but the last rounding
    fast = dt == BF and dk >= 64 and L > 16
    assert err <= (4 * 2.0 ** -8 if fast else G.tol32(L, dk, "grad")), err


def test_layer_without_widening():
    """An autograd layer that hands the gates' gradient on as it is."""
    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, beta, g):
            ctx.save_for_backward(q, k, v, beta, g)
            return efla.efla_gated_chunk_fwd(q, k, v, beta, g, want_final=False)[0]

        @staticmethod
        def backward(ctx, do):
            return efla.efla_gated_chunk_bwd(*ctx.saved_tensors, do.contiguous(), want_ds0=False, dg_dtype=F32)[:5]

    x = R.slow(1, 130, 4, 2, 64, 64, BF, seed=5)
    leaves = [x[n].cuda().requires_grad_() for n in G.NAMES]
    o = Layer.apply(*leaves)
    o.float().square().sum().mul(0.5).backward()
    assert leaves[4].grad.dtype == F32
    want = efla.efla_gated_chunk_bwd(*(t.detach() for t in leaves), o.detach(), dg_dtype=F32)
    for a, b in zip(leaves, want):
        assert torch.equal(a.grad, b)
