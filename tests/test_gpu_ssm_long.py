"""The scan at lengths of dozens of chunks: segments of three chunks and more in the forward
pass, gradients of 2048 tokens; and states, which are float32, held to float32."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def dev(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def ins(x):
    return [x[n] for n in ("q", "k", "v", "dt", "a")], dict(d=x["d"], dt_bias=x["bias"])


def workspace(slots, H, dk, dv):
    """Of `slots` segments a head: their states and their decays, each to whole 256 bytes."""
    return sum((slots * H * n * 4 + 255) // 256 * 256 for n in (dk * dv, 1))


# (sequences, tokens, heads, key heads, d_k, d_v, type, chunks a segment): heads and value blocks that leave four segments
# a sequence (two for the pairs) to be wanted
CUTS = [(1, 760, 16, 4, 128, 128, BF, 3), (1, 1000, 32, 1, 64, 64, BF, 4), (1, 1100, 16, 16, 128, 128, BF, 5),
        (1, 1760, 32, 8, 128, 64, BF, 7), (1, 2048, 16, 1, 128, 128, BF, 8), (1, 2999, 16, 4, 64, 128, BF, 12),
        (2, 2113, 16, 2, 64, 64, BF, 9), (1, 380, 16, 4, 64, 64, F32, 3), (1, 1024, 16, 1, 128, 64, F32, 8),
        (1, 700, 32, 4, 16, 32, BF, 6), (2, 600, 16, 16, 32, 32, F32, 5)]


@pytest.mark.parametrize("B,L,H,Hk,dk,dv,dtype,per", CUTS)
def test_dense_segments(B, L, H, Hk, dk, dv, dtype, per):
    C = 64 if dtype == BF and dk >= 64 and dv >= 32 else 32
    assert efla.efla_ssm_fwd_workspace_size(B, H, Hk, L, dk, dv, dtype) == workspace(B * -(-L // (per * C)), H, dk, dv)
    for s0 in (True, False):
        x = dev(R.make_scan(B, L, H, Hk, dk, dv, dtype, seed=L, s0=s0, steps=(1e-4, 0.1)))
        a, kw = ins(x)
        o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        ro, rs = R.scan_ref(*R.wide(x))
        assert R.rel(o, ro) <= R.tol_o(dtype, L, dk) and R.rel(S, rs) <= R.tol_s(dtype, L, dk)
        if s0:
            st = x["s0"].clone()
            o2, S2 = efla.efla_ssm_fwd(*a, s0=st, s_final=st, **kw)
            assert S2 is st and torch.equal(o, o2) and torch.equal(S, st)


@pytest.mark.parametrize("lens,H,dk,dv,dtype,per", [
    ([2100, 900], 16, 64, 64, BF, 6), ([0, 2990, 10], 8, 128, 64, BF, 3), ([1500, 0, 1400, 1], 4, 64, 128, BF, 3),
    ([5000], 32, 128, 64, BF, 20), ([3, 1000], 8, 64, 64, F32, 4), ([1999, 2000], 8, 128, 128, BF, 8)])
def test_packed_segments(lens, H, dk, dv, dtype, per):
    N, T, Hk = len(lens), sum(lens) + 3, 2
    C = 64 if dtype == BF else 32
    assert efla.efla_ssm_fwd_varlen_workspace_size(N, H, Hk, T, dk, dv, dtype) == workspace(T // (per * C) + N, H, dk, dv)
    x = dev(R.make_scan(N + 2, 0, H, Hk, dk, dv, dtype, lead=(T,), steps=(1e-4, 0.1)))
    a, kw = ins(x)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    slots = torch.arange(N, 0, -1, dtype=torch.int32)
    pool, o = x["s0"].clone(), torch.full((T, H, dv), 3.0, dtype=dtype, device="cuda")
    efla.efla_ssm_fwd_varlen(*a, cu, s0=pool, slots=slots.cuda(), o=o, s_final=pool, **kw)
    at = 0
    for n, slot in zip(lens, slots.tolist()):
        part = {m: x[m][None, at:at + n] for m in ("q", "k", "v", "dt")}
        part.update({m: x[m] for m in ("a", "d", "bias")}, s0=x["s0"][slot:slot + 1])
        ro, rs = R.scan_ref(*R.wide(part))
        if n:
            assert R.rel(o[None, at:at + n], ro) <= R.tol_o(dtype, n, dk)
        assert R.rel(pool[slot:slot + 1], rs) <= R.tol_s(dtype, n, dk)
        at += n
    assert bool((o[at:] == 3.0).all()) and torch.equal(pool[0], x["s0"][0]) and torch.equal(pool[N + 1], x["s0"][N + 1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L,H,Hk,dk,dv", [(2048, 4, 2, 64, 64), (2031, 2, 1, 128, 128), (1537, 3, 3, 128, 64)])
def test_gradients_of_a_layers_length(dtype, L, H, Hk, dk, dv):
    x = dev(R.make_scan(1, L, H, Hk, dk, dv, dtype, seed=L, steps=(1e-4, 0.1)))
    a, kw = ins(x)
    gen = torch.Generator().manual_seed(L)
    d_o = torch.randn(1, L, H, dv, generator=gen).to(dtype).cuda()
    dsf = torch.randn(1, H, dk, dv, generator=gen).cuda()
    got = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], ds_final=dsf, **kw)
    want, scale = R.scan_grads_ref(x, d_o, dsf)
    for name, y in zip(R.GRADS, got):
        err = R.rel(y, want[name], scale.get(name))
        assert err <= R.tol_grad(dtype, L, dk, name), (name, err)
    again = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], ds_final=dsf, **kw)
    assert all(torch.equal(p, r) for p, r in zip(got, again))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rate", [-16.0, -1.0])
def test_rate_gradient_of_a_layers_length(dtype, rate):
    """As test_rate_gradient_of_neighbours: 32 half steps of the root of the terms' summed squares."""
    L = 2048
    x = R.make_scan(2, L, 4, 2, 64, 64, dtype, seed=L, s0=False, steps=(0.05, 0.1))
    x["q"], x["k"] = x["q"].abs(), x["k"].abs()
    x["a"].fill_(rate)
    a, kw = ins(dev(x))
    d_o = torch.randn(2, L, 4, 64, generator=torch.Generator().manual_seed(L)).to(dtype)
    da = efla.efla_ssm_bwd(*a, d_o.cuda(), **kw)[4].double().cpu()
    want, scale = R.rate_gradient_ref(x, d_o)
    assert bool(((da - want).abs() <= 32 * 2.0 ** -24 * scale).all()), ((da - want) / scale * 2.0 ** 24).tolist()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [1, 2, 7, 15, 17, 31, 63, 64, 65, 100, 128])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 32)])
def test_states_are_float32(dtype, L, dk, dv):
    """S from no state and ds0 from no final gradient, so that neither starts with values that have no error.  A term of
    either has about four roundings of its factors (the step, its exponential, their product, the product's parts), each
    a half step 2^-24, and their sum over up to 128 tokens a random walk of sqrt(128) more: 16 half steps.  In two bf16
    parts in place of three a factor would be off by 2^-18 / sqrt(3), 37 half steps."""
    x = dev(R.make_scan(2, L, 4, 2, dk, dv, dtype, seed=L, s0=False))
    a, kw = ins(x)
    _, S = efla.efla_ssm_fwd(*a, **kw)
    _, rs = R.scan_ref(*R.wide(x))
    d_o = torch.randn(2, L, 4, dv, generator=torch.Generator().manual_seed(L)).to(dtype).cuda()
    ds0 = efla.efla_ssm_bwd(*a, d_o, **kw)[7]
    q = x["q"].double().repeat_interleave(2, 2)
    D = R.softplus(x["dt"].double() + x["bias"].double())
    e = torch.exp(x["a"].double() * D.cumsum(1))
    want = ((e[..., None] * q)[..., None] * d_o.double()[..., None, :]).sum(1)
    assert R.rel(S, rs) <= 16 * 2.0 ** -24, R.rel(S, rs) * 2.0 ** 24
    assert R.rel(ds0, want) <= 16 * 2.0 ** -24, R.rel(ds0, want) * 2.0 ** 24


@pytest.mark.parametrize("L", [32, 64, 129])
def test_pairs_behind_a_reset(L):
    """Float32 outputs behind a token in every chunk that decays by e^-128: o's terms have the roundings of a dot product
    over 64, a random walk of 8 half steps, and of the factors and the sum over the tokens, 16 in all.  The exponent
    as one float, between 2^7 and 2^8 in log2 units, would be off by up to 2^-17, the pairs' decays by up to 88 half steps."""
    x = R.make_scan(2, L, 4, 2, 64, 64, F32, seed=L, s0=False)
    x["a"].fill_(-16.0)
    x["dt"][:, 2::32] = 8.0 - x["bias"]  # D of 8
    x["d"].zero_()
    late = torch.arange(L) % 32 > 4
    a, kw = ins(dev(x))
    o, _ = efla.efla_ssm_fwd(*a, **kw)
    ro, _ = R.scan_ref(*R.wide(x))
    assert R.rel(o.cpu()[:, late], ro[:, late]) <= 16 * 2.0 ** -24, R.rel(o.cpu()[:, late], ro[:, late]) * 2.0 ** 24
