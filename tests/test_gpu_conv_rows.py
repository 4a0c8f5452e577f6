"""The convolution's outputs beside its inputs in the rows of one tensor, and over them."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,D", [(2, 90, 64), (3, 1, 8), (1, 300, 33)])
def test_outputs_beside_inputs(dtype, B, L, D):
    x = {n: t.cuda() for n, t in R.make_conv(B, L, D, 4, dtype).items()}
    dy = torch.randn(B, L, D, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    want, fin = efla.efla_conv_fwd(x["x"], x["w"], x["bias"], x["s0"])
    grads = efla.efla_conv_bwd(x["x"], x["w"], dy, x["bias"], x["s0"])
    rows = torch.full((B, L, 4 * D), 7.0, dtype=dtype, device="cuda")
    rows[..., D:2 * D], rows[..., 2 * D:3 * D] = x["x"], dy
    inp, gy = rows[..., D:2 * D], rows[..., 2 * D:3 * D]
    y, f = efla.efla_conv_fwd(inp, x["w"], x["bias"], x["s0"], y=rows[..., :D])
    assert torch.equal(y, want) and torch.equal(f, fin)
    got = efla.efla_conv_bwd(inp, x["w"], gy, x["bias"], x["s0"], dx=rows[..., 3 * D:])
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert torch.equal(inp, x["x"]) and torch.equal(gy, dy) and torch.equal(rows[..., :D], want)


def test_outputs_over_inputs():
    x = {n: t.cuda() for n, t in R.make_conv(2, 50, 64, 4, BF).items()}
    dy, cu = torch.randn_like(x["x"]), torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    keep = x["x"].clone()
    with pytest.raises(efla.EflaError):
        efla.efla_conv_fwd(x["x"], x["w"], y=x["x"])
    with pytest.raises(efla.EflaError):
        efla.efla_conv_fwd_varlen(x["x"][0], x["w"], cu, y=x["x"][0])
    for dx in (x["x"], dy):
        with pytest.raises(efla.EflaError):
            efla.efla_conv_bwd(x["x"], x["w"], dy, dx=dx)
    assert torch.equal(x["x"], keep)
    state, other = x["s0"].clone(), x["s0"].clone()  # a token's row is read and written by one lane
    row = x["x"][:, 0].clone()
    want = efla.efla_conv_step(row, x["w"], state, x["bias"])
    got = efla.efla_conv_step(row, x["w"], other, x["bias"], y=row)
    assert got is row and torch.equal(row, want) and torch.equal(state, other)
