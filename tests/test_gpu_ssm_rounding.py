"""The rate's gradient over many tokens whose queries, keys and values are behind a SiLU,
mostly of one sign: rounding errors that all go one way would add up over them."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L,dk,dv", [(256, 64, 64), (1024, 128, 128), (2048, 128, 128), (2048, 64, 32), (2048, 128, 64)])
@pytest.mark.parametrize("rates", [(-16.0, -1.0), (-2.0, -0.1)])
def test_rate_gradient_of_positive_inputs(dtype, L, dk, dv, rates):
    """A pair's term of da has the roundings of two dot products, a random walk of sqrt(64) to sqrt(128) half steps, and of
    the factors; states and their gradients, which the pairs of different chunks go through, the same again: 32 half
    steps of the root of the terms' summed squares, at any length."""
    B, H, Hk = 2, 8, 4
    x = R.make_scan(B, L, H, Hk, dk, dv, dtype, s0=False)
    gen = torch.Generator().manual_seed(L + dv)
    for n in ("q", "k", "v"):
        t = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        x[n] = (t * torch.sigmoid(t)).to(dtype)
    x["a"] = torch.linspace(*rates, H)
    d_o = torch.randn(x["v"].shape, generator=gen).to(dtype).cuda()
    x = {n: None if t is None else t.cuda() for n, t in x.items()}
    da = efla.efla_ssm_bwd(*(x[n] for n in ("q", "k", "v", "dt", "a")), d_o, x["d"], x["bias"])[4].double()
    want, scale = R.rate_gradient_ref(x, d_o)
    assert bool(((da - want).abs() <= 32 * 2.0 ** -24 * scale).all()), ((da - want) / scale * 2.0 ** 24).tolist()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_states_of_a_slow_head(dtype):
    """A state that forgets little.  Float32: 64 chunks of 32 tokens, whose own sums are added with one rounding each, and
    whose decays are rounded too, and a random walk of 64 in the sums: sqrt(192) roundings of a half step / sqrt(3), 8 half
    steps in the 2-norm; half of that again is allowed.  bf16: 32 chunks of 64 tokens, six products of each added to the
    state itself and rounded down, up to a half step each: 96, and the 8."""
    x = R.make_scan(8, 2048, 16, 1, 64, 64, dtype, s0=False)  # sequences and heads enough not to be cut into segments
    assert efla.efla_ssm_fwd_workspace_size(8, 16, 1, 2048, 64, 64, dtype) == 0
    x["a"].fill_(-1e-4)
    x = {n: None if t is None else t.cuda() for n, t in x.items()}
    _, S = efla.efla_ssm_fwd(*(x[n] for n in ("q", "k", "v", "dt", "a")), x["d"], x["bias"])
    D = R.softplus(x["dt"].double() + x["bias"].double())
    G = (x["a"].double() * D).cumsum(1)
    w = (torch.exp(G[:, -1:] - G) * D)[0]
    want = torch.stack([x["k"][0, :, 0].double().t().contiguous() @ (w[:, h, None] * x["v"][0, :, h].double()) for h in range(16)])
    assert R.rel(S[0], want) <= (104 if dtype == BF else 12) * 2.0 ** -24
