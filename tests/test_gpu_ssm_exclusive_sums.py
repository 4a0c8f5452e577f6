"""The rate's gradient takes the tokens before a step alone: a last token whose own term
is far larger than theirs does not enter it, nor its rounding."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [2, 20, 32, 64, 100])
@pytest.mark.parametrize("rate", [-16.0, -1.0])
def test_a_large_last_token(dtype, L, rate):
    """With dO = 0 and dLoss/dS_L = X, from no state,
        da = sum_j (C_L - C_j) p_j,   p_j = e^{a (C_L - C_j)} D_j k_j . (X v_j),   C_j = D_1 + .. + D_j.
    A product's term has the roundings of sums over 64 and 64 values and of the factors, 32 half steps of the root of
    its summed squares with the parts of X; the sums over tokens six levels each of a prefix and of a tree, 12 half
    steps of the absolute sum.  The last token's p, 2^20 times the others, has the factor zero."""
    B, H, Hk, d = 2, 4, 2, 64
    x = R.make_scan(B, L, H, Hk, d, d, dtype, seed=L, s0=False, steps=(0.05, 0.1))
    x["v"][:, -1] *= 2.0 ** 20
    x["a"].fill_(rate)
    X = torch.randn(B, H, d, d, generator=torch.Generator().manual_seed(L))
    dev = {n: None if t is None else t.cuda() for n, t in x.items()}
    da = efla.efla_ssm_bwd(*(dev[n] for n in ("q", "k", "v", "dt", "a")), torch.zeros_like(dev["v"]), dev["d"], dev["bias"],
                           ds_final=X.cuda())[4].double().cpu()
    _, k, v, dt, a, _, bias, _ = R.wide(x)
    k, v = k.repeat_interleave(H // Hk, 2).transpose(1, 2), v.transpose(1, 2)
    D = R.softplus(dt + bias).transpose(1, 2)
    after = D.flip(-1).cumsum(-1).flip(-1) - D
    after[..., -1] = 0
    f = after * torch.exp(a[:, None] * after) * D
    term = f * (k * (v @ X.double().transpose(-1, -2))).sum(-1)
    squares = (f * f * (k * k * ((v * v) @ (X.double() ** 2).transpose(-1, -2))).sum(-1)).sum((0, 2)).sqrt()
    bound = 2.0 ** -24 * (32 * squares + 12 * term.abs().sum((0, 2)))
    assert bool(((da - term.sum((0, 2))).abs() <= bound).all()), ((da - term.sum((0, 2))) / bound).tolist()
