"""The gated delta rule on the GPU where its states outlive a chunk many times over,
and where keys are far from unit length (tests/_gated_regimes.py has the inputs;
tests/_gated.py the 64-bit form and the tolerances; tests/test_gated_regimes.py
shows that the first see a lost carry)."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _gated as G
from tests import _gated_regimes as R
from tests.test_gpu_gated import GRADS, dev, grads_ref, ids

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

SLOW = [(1, 321, 4, 2, 128, 128, BF, "exact"), (2, 321, 4, 4, 64, 64, BF, "euler"), (1, 200, 8, 2, 64, 128, BF, "exact"),
        (2, 200, 4, 1, 128, 64, BF, "euler"), (1, 170, 4, 4, 64, 64, BF, "exact"), (1, 200, 4, 2, 32, 32, BF, "exact"),
        (1, 321, 4, 4, 64, 64, F32, "exact"), (1, 200, 4, 2, 128, 128, F32, "euler"), (2, 333, 4, 2, 64, 128, F32, "exact"),
        (1, 321, 4, 1, 32, 32, F32, "euler"), (30, 150, 4, 4, 64, 64, F32, "exact")]


@pytest.mark.parametrize("p", SLOW, ids=ids)
def test_slow_heads_forward(p):
    B, L, H, Hk, dk, dv, dt, rule = p
    x = R.slow(B, L, H, Hk, dk, dv, dt, seed=L + dk)
    a = dev(x)
    o, S = efla.efla_gated_chunk_fwd(*(a[n] for n in G.NAMES), a["s0"], rule=rule)
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double(), rule)
    eo, es = G.rel(o, wo), G.rel(S, wS)
    print(f"slow {ids(p)}: o {eo:.2e} of {G.tol_o(dt, L, dk):.2e}, S {es:.2e} of {G.tol_s(dt, L, dk):.2e}", flush=True)
    assert eo <= G.tol_o(dt, L, dk) and es <= G.tol_s(dt, L, dk)


@pytest.mark.parametrize("p", SLOW[:-1], ids=ids)
def test_slow_heads_backward(p):
    B, L, H, Hk, dk, dv, dt, rule = p
    x = R.slow(B, L, H, Hk, dk, dv, dt, seed=L + dk)
    gen = torch.Generator().manual_seed(77)
    do, dsf = torch.randn(B, L, H, dv, generator=gen).to(dt), torch.randn(B, H, dk, dv, generator=gen)
    a = dev(x)
    got = efla.efla_gated_chunk_bwd(*(a[n] for n in G.NAMES), do.cuda(), a["s0"], dsf.cuda(), rule=rule)
    errs = {n: G.rel(g, w) for n, g, w in zip(GRADS, got, grads_ref(x, do, dsf, rule))}
    print(f"slow {ids(p)}: " + ", ".join(f"{n} {e:.2e}" for n, e in errs.items()) + f" of {G.tol_grad(dt, L, dk):.2e}", flush=True)
    assert all(e <= G.tol_grad(dt, L, dk) for e in errs.values()), errs


@pytest.mark.parametrize("H,Hk,dk,dv,dt", [(4, 2, 128, 128, BF), (4, 4, 64, 64, BF), (4, 1, 64, 128, F32), (4, 2, 128, 64, F32)], ids=str)
def test_slow_heads_packed(H, Hk, dk, dv, dt):
    lens = [300, 1, 129, 0, 64, 200]
    T = sum(lens)
    x = R.slow(len(lens), 0, H, Hk, dk, dv, dt, seed=T + dk, lead=(T,))
    a = dev(x)
    p = efla.efla_pack_plan(torch.tensor(lens, dtype=torch.int32).cuda(), T)
    o, S = efla.efla_gated_chunk_fwd_varlen(*(a[n] for n in G.NAMES), p.cu_seqlens, a["s0"], order=p.order)
    at = 0
    for i, n in enumerate(lens):
        wo, wS = G.forward_ref(*(t[None, at:at + n] for t in G.wide(x)), x["s0"][i:i + 1].double())
        assert n == 0 or G.rel(o[at:at + n], wo[0]) <= G.tol_o(dt, n, dk)
        assert G.rel(S[i], wS[0]) <= G.tol_s(dt, n, dk)
        at += n


def test_extreme_gates_need_no_slack():
    """The gates of test_forward_extreme_gates: their sums are held in 64 bits, so the tolerances
    of ordinary gates hold (P's factors, from 32-bit sums, are far below P's own rounding to bf16)."""
    L = 200
    for dt in (F32, BF):
        for d in (32, 64, 128):
            x = G.make(1, L, 2, 2, d, d, dt, seed=6, decay=2.0)
            g = x["g"]
            g[:, 5], g[:, 70], g[:, 71] = float("-inf"), torch.finfo(F32).min, float("-inf")
            g[:, 100:110], g[:, 110:120] = 0.0, 0.05
            g[:, 199] = -300.0
            a = dev(x)
            o, S = efla.efla_gated_chunk_fwd(*(a[n] for n in G.NAMES), a["s0"])
            wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
            assert G.rel(o, wo) <= G.tol_o(dt, L, d) and G.rel(S, wS) <= G.tol_s(dt, L, d), (dt, d)


LAM = [10, 100, 1000, "spread"]


@pytest.mark.parametrize("lam", LAM)
@pytest.mark.parametrize("d,dt", [(64, BF), (128, BF), (32, F32), (64, F32), (128, F32)], ids=str)
def test_long_and_zero_keys(d, dt, lam):
    """The exact rule keeps 0 <= alpha |k|^2 <= 1 at every key length, so the forward's tolerances hold as they
    are.  dbeta alone is conditioned by x = beta |k|^2: its factor e^{-x} takes up x's own relative error, |k|^2
    being a float32 sum of d_k squares (sqrt(d_k) + 2 roundings of 2^-24), by which its tolerance grows.  (Autograd
    forms that factor as expm1(-x) + 1: zero from x = 37 on, where the kernel's e^{-x} must be below 1e-15.)"""
    B, L, H, Hk = 1, 200, 4, 2
    x = R.stiff(B, L, H, Hk, d, d, dt, d + L, lam)
    a = dev(x)
    args = [a[n] for n in G.NAMES]
    o, S = efla.efla_gated_chunk_fwd(*args, a["s0"])
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
    errs = {"o": (G.rel(o, wo), G.tol_o(dt, L, d)), "S": (G.rel(S, wS), G.tol_s(dt, L, d))}
    gen = torch.Generator().manual_seed(5)
    do, dsf = torch.randn(B, L, H, d, generator=gen).to(dt), torch.randn(B, H, d, d, generator=gen)
    got = efla.efla_gated_chunk_bwd(*args, do.cuda(), a["s0"], dsf.cuda())
    top = 1000 if lam == "spread" else lam
    for n, g, w in zip(GRADS, got, grads_ref(x, do, dsf, "exact")):
        extra = top * (d ** 0.5 + 2) * 2.0 ** -24 if n == "dbeta" else 0.0
        errs[n] = (G.rel(g, w), G.tol_grad(dt, L, d) + extra)
    print(f"lam {lam} d {d} {dt}: " + ", ".join(f"{n} {e:.2e}/{t:.1e}" for n, (e, t) in errs.items()), flush=True)
    assert all(e <= t for e, t in errs.values()), errs


@pytest.mark.parametrize("lam", LAM)
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_step_with_long_and_zero_keys(dt, lam):
    x = R.stiff(3, 6, 4, 2, 64, 64, dt, 3, lam)
    a = dev(x)
    st = a["s0"].clone()
    outs = [efla.efla_gated_step(*(a[n][:, t].contiguous() for n in G.NAMES), st) for t in range(6)]
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
    assert G.rel(torch.stack(outs, 1), wo) <= G.tol32(6, 64) + (0 if dt == F32 else 2.0 ** -8)
    assert G.rel(st, wS) <= G.tol32(6, 64)


@pytest.mark.parametrize("d,dt", [(64, BF), (128, BF), (32, F32), (64, F32)], ids=str)
def test_growing_gates(d, dt):
    """Positive gates: a state that grows by e^40 over the sequence, e^19 a chunk.  Exponents of gate differences are
    then positive, up to 0.3 x 63 = 19: a float32 exponential of it is off by 19 x 2^-24 more, which each token's
    factor passes on once; gradients pass two such factors."""
    L = 130
    x = G.make(1, L, 4, 2, d, d, dt, seed=d)
    gen = torch.Generator().manual_seed(2)
    x["g"] = 0.3 + 0.01 * torch.randn(x["g"].shape, generator=gen)
    do, dsf = torch.randn(1, L, 4, d, generator=gen).to(dt), torch.randn(1, 4, d, d, generator=gen)
    a = dev(x)
    args = [a[n] for n in G.NAMES]
    o, S = efla.efla_gated_chunk_fwd(*args, a["s0"])
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
    more = 20 * 2.0 ** -24 * L ** 0.5
    errs = {"o": (G.rel(o, wo), G.tol_o(dt, L, d) + more), "S": (G.rel(S, wS), G.tol_s(dt, L, d) + more)}
    got = efla.efla_gated_chunk_bwd(*args, do.cuda(), a["s0"], dsf.cuda())
    for n, g, w in zip(GRADS, got, grads_ref(x, do, dsf, "exact")):
        errs[n] = (G.rel(g, w), G.tol_grad(dt, L, d) + 2 * more)
    print(f"growth d {d} {dt}: " + ", ".join(f"{n} {e:.2e}/{t:.1e}" for n, (e, t) in errs.items()), flush=True)
    assert all(e <= t for e, t in errs.values()), errs


@pytest.mark.parametrize("d,dt", [(128, BF), (64, BF), (64, F32)], ids=str)
def test_long_sequences_of_slow_heads(d, dt):
    """2048 tokens, the first head without any decay (the 64-bit form on the GPU)."""
    L, H = 2048, 2
    x = R.slow(1, L, H, 1, d, d, dt, seed=d)
    gen = torch.Generator().manual_seed(2)
    do, dsf = torch.randn(1, L, H, d, generator=gen).to(dt).cuda(), torch.randn(1, H, d, d, generator=gen).cuda()
    a = dev(x)
    args = [a[n] for n in G.NAMES]
    o, S = efla.efla_gated_chunk_fwd(*args, a["s0"])
    leaves = [t.requires_grad_() for t in (*G.wide(a), a["s0"].double())]
    wo, wS = G.forward_ref(*leaves)
    errs = {"o": (G.rel(o, wo), G.tol_o(dt, L, d)), "S": (G.rel(S, wS), G.tol_s(dt, L, d))}
    want = torch.autograd.grad((wo * do.double()).sum() + (wS * dsf.double()).sum(), leaves)
    got = efla.efla_gated_chunk_bwd(*args, do, a["s0"], dsf)
    for n, g, w in zip(GRADS, got, want):
        errs[n] = (G.rel(g, w), G.tol_grad(dt, L, d))
    print(f"long d {d} {dt}: " + ", ".join(f"{n} {e:.2e}/{t:.1e}" for n, (e, t) in errs.items()), flush=True)
    assert all(e <= t for e, t in errs.values()), errs
