"""The gated entry points where they can go wrong besides the ordinary cases of
tests/test_gpu_gated.py: resets, infinite values behind them, the sizes at which
another kernel takes over, side streams, many sequences, malformed tables, and
tensors past 2^32 bytes (tolerances: tests/_gated.py)."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _gated as G
from tests.test_gpu_gated import GRADS, dev, grads_ref, ids

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
RESET = float("-inf")


def with_resets(L, H, Hk, d, dt, seed):
    """Resets at every third token, the last 16 tokens of L plain: the sums of gates
    reach -128 L / 3 while the gates that matter for the last state are small."""
    x = G.make(1, L, H, Hk, d, d, dt, seed=seed, decay=0.05)
    x["g"][:, :L - 15:3] = RESET
    return x


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
@pytest.mark.parametrize("d", [32, 64, 128])
def test_resets_cost_no_accuracy(dt, d):
    L = 64 * 3
    x = with_resets(L, 2, 2, d, dt, 5)
    a = dev(x)
    o, S = efla.efla_gated_chunk_fwd(*(a[n] for n in G.NAMES), a["s0"])
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
    # as a sequence of its own from the last reset on: 18 tokens, one or two chunks
    assert G.rel(o, wo) <= G.tol_o(dt, 18, d) and G.rel(S, wS) <= G.tol_s(dt, 18, d)
    # and nothing before it has any influence: those tokens left out, the same to the same tolerance
    cut = (L - 16) // 3 * 3
    o2, S2 = efla.efla_gated_chunk_fwd(*(a[n][:, cut:].contiguous() for n in G.NAMES))
    assert G.rel(S2, S) <= 2 * G.tol_s(dt, 18, d) and G.rel(o2, o[:, cut:]) <= 2 * G.tol_o(dt, 18, d)


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
@pytest.mark.parametrize("d", [32, 64])
def test_backward_with_resets(dt, d):
    L = 128
    x = with_resets(L, 2, 1, d, dt, 6)
    gen = torch.Generator().manual_seed(2)
    do, dsf = torch.randn(1, L, 2, d, generator=gen).to(dt), torch.randn(1, 2, d, d, generator=gen)
    a = dev(x)
    got = efla.efla_gated_chunk_bwd(*(a[n] for n in G.NAMES), do.cuda(), a["s0"], dsf.cuda())
    want = grads_ref(x, do, dsf, "exact")
    for name, p, r in zip(GRADS, got, want):
        assert bool(torch.isfinite(p).all()), name
        # the first token resets the state: no gradient reaches s0
        assert (not bool(p.any())) if name == "ds0" else G.rel(p, r) <= G.tol_grad(dt, 18, d), name


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
def test_step_reset_takes_a_finite_state_to_zero(dt):
    x = G.make(1, 1, 2, 2, 64, 64, dt, seed=7)
    x["g"][:] = RESET
    a = dev(x)
    st = (torch.rand(1, 2, 64, 64) * 1e30).cuda()
    o = efla.efla_gated_step(*(a[n][:, 0].contiguous() for n in G.NAMES), st)
    wo, wS = G.forward_ref(*G.wide(x))
    assert G.rel(o, wo[:, 0]) <= G.tol_o(dt, 1, 64) and G.rel(st, wS) <= G.tol32(1, 64)


# L at which the forward changes kernels (d 64 and 128, few and many workgroups), and the backward
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,L", [(1, 15), (1, 16), (1, 17), (1, 31), (1, 32), (1, 33), (1, 48), (1, 65),
                                 (1, 112), (1, 113), (1, 176), (1, 177), (20, 1), (20, 47), (20, 49), (20, 64), (20, 65), (20, 127),
                                 (70, 8), (70, 24), (130, 3)])
def test_where_kernels_change(B, L, d):
    x = G.make(B, L, 4, 2, d, d, BF, seed=L)
    a = dev(x)
    args = [a[n] for n in G.NAMES]
    o, S = efla.efla_gated_chunk_fwd(*args, a["s0"])
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
    assert G.rel(o, wo) <= G.tol_o(BF, L, d) and G.rel(S, wS) <= G.tol_s(BF, L, d)
    if B > 1:
        return
    do = torch.randn(B, L, 4, d, generator=torch.Generator().manual_seed(1)).to(BF)
    got = efla.efla_gated_chunk_bwd(*args, do.cuda(), a["s0"])
    for name, p, r in zip(GRADS, got, grads_ref(x, do, None, "exact")):
        assert G.rel(p, r) <= G.tol_grad(BF, L, d), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,L", [(1, 31), (1, 32), (2, 47), (1, 333), (30, 100), (30, 161), (12, 200)])
def test_fp32_where_kernels_change(B, L, d):
    x = G.make(B, L, 6, 3, d, d, F32, seed=L)
    a = dev(x)
    args = [a[n] for n in G.NAMES]
    o, S = efla.efla_gated_chunk_fwd(*args, a["s0"], rule="euler")
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double(), "euler")
    assert G.rel(o, wo) <= G.tol_o(F32, L, d) and G.rel(S, wS) <= G.tol_s(F32, L, d)
    if B == 1:
        do = torch.randn(B, L, 6, d, generator=torch.Generator().manual_seed(1))
        got = efla.efla_gated_chunk_bwd(*args, do.cuda(), a["s0"], chunk=16, rule="euler")
        for name, p, r in zip(GRADS, got, grads_ref(x, do, None, "euler")):
            assert G.rel(p, r) <= G.tol_grad(F32, L, d), name


@pytest.mark.parametrize("chunk", [16, 32, 64])
@pytest.mark.parametrize("dt", [F32, BF], ids=str)
def test_chunk_does_not_matter(dt, chunk):
    x = G.make(1, 100, 2, 2, 64, 64, dt, seed=4)
    a = dev(x)
    args = [a[n] for n in G.NAMES]
    do = torch.randn(1, 100, 2, 64, generator=torch.Generator().manual_seed(1)).to(dt)
    o, S = efla.efla_gated_chunk_fwd(*args, a["s0"], chunk=chunk)
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
    assert G.rel(o, wo) <= G.tol_o(dt, 100, 64) and G.rel(S, wS) <= G.tol_s(dt, 100, 64)
    got = efla.efla_gated_chunk_bwd(*args, do.cuda(), a["s0"], chunk=chunk)
    for name, p, r in zip(GRADS, got, grads_ref(x, do, None, "exact")):
        assert G.rel(p, r) <= G.tol_grad(dt, 100, 64), name


def test_final_state_in_place():
    for dt, L in ((BF, 130), (BF, 20), (F32, 130), (BF, 0)):
        x = dev(G.make(2, L, 4, 2, 64, 64, dt, seed=3))
        a = [x[n] for n in G.NAMES]
        o, S = efla.efla_gated_chunk_fwd(*a, x["s0"])
        st = x["s0"].clone()
        o2, S2 = efla.efla_gated_chunk_fwd(*a, st, s_final=st)
        assert S2 is st and torch.equal(S, st) and torch.equal(o, o2)


def test_side_stream_order():
    """Inputs written on the call's own stream just before it, outputs read there just after."""
    H, d, L = 4, 128, 200
    x = dev(G.make(1, L, H, H, d, d, BF, seed=2))
    src = [x[n] for n in G.NAMES]
    do = torch.randn(1, L, H, d, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    want = [*efla.efla_gated_chunk_fwd(*src, x["s0"]), *efla.efla_gated_chunk_bwd(*src, do, x["s0"])]
    big = torch.randn(8192, 8192).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = [torch.zeros_like(t) for t in src]
        big = big @ big  # some milliseconds
        for t, u in zip(a, src):
            t.copy_(u)
        got = [*efla.efla_gated_chunk_fwd(*a, x["s0"]), *efla.efla_gated_chunk_bwd(*a, do, x["s0"])]
        lens = torch.full((1,), L, dtype=torch.int32).cuda()
        p = efla.efla_pack_plan(lens, L)
        o, S = efla.efla_gated_chunk_fwd_varlen(*(t[0] for t in a), p.cu_seqlens, x["s0"], order=p.order)
        got = [t.clone() for t in (*got, o[None], S)]
    s.synchronize()
    for p, q in zip(got, want + want[:2]):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dt,d", [(BF, 64), (F32, 16)], ids=str)
def test_many_sequences(dt, d):
    """More sequences than one workgroup ranks, most of them of no or one token."""
    N = 4200
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 3, (N,), generator=gen, dtype=torch.int32)
    lens[7], lens[4100] = 300, 130
    T = int(lens.sum())
    x = G.make(N, 0, 1, 1, d, d, dt, seed=9, lead=(T,))
    a = dev(x)
    p = efla.efla_pack_plan(lens.cuda(), T + 5)
    args = [torch.cat([a[n], torch.full_like(a[n][:5], float("nan"))]) for n in G.NAMES]  # rows of no sequence
    o = torch.full((T + 5, 1, d), 7.0, dtype=dt).cuda()
    o, S = efla.efla_gated_chunk_fwd_varlen(*args, p.cu_seqlens, a["s0"], order=p.order, o=o)
    assert bool((o[T:] == 7).all())
    o2, S2 = efla.efla_gated_chunk_fwd_varlen(*args, p.cu_seqlens, a["s0"])
    assert torch.equal(o[:T], o2[:T]) and torch.equal(S, S2)
    cu = [0, *lens.cumsum(0).tolist()]
    empty = [u for u in range(N) if lens[u] == 0]
    assert torch.equal(S[empty], a["s0"][empty])
    for u in (7, 4100, *[u for u in range(0, N, 97) if lens[u] > 0]):
        w = [t[cu[u]:cu[u + 1]][None] for t in G.wide(x)]
        wo, wS = G.forward_ref(*w, x["s0"][u:u + 1].double())
        n = int(lens[u])
        assert G.rel(o[cu[u]:cu[u + 1]], wo[0]) <= G.tol_o(dt, n, d) and G.rel(S[u], wS[0]) <= G.tol_s(dt, n, d)


def test_malformed_tables_stay_in_range():
    """Offsets that fall, start below zero or pass T, an order that is no permutation, slots without a row."""
    T, H, d = 200, 2, 64
    for dt in (BF, F32):
        x = dev(G.make(4, 0, H, H, d, d, dt, seed=2, lead=(T,)))
        a = [x[n] for n in G.NAMES]
        guard = torch.full((3, T, H, d), 5.0, dtype=dt).cuda()
        pool = torch.full((6, 4, H, d, d), 5.0).cuda()
        for cu in ([-5, 50, 30, 120, 999], [0, 2 ** 31 - 1, -2 ** 31, 100, 200], [200, 200, 200, 200, 200]):
            efla.efla_gated_chunk_fwd_varlen(*a, torch.tensor(cu, dtype=torch.int32).cuda(), pool[2], o=guard[1],
                                             slots=torch.tensor([0, 7, -3, 2 ** 31 - 1], dtype=torch.int32).cuda(),
                                             order=torch.tensor([9, -1, 2, 2], dtype=torch.int32).cuda(), s_final=pool[2])
        torch.cuda.synchronize()
        assert bool((guard[0] == 5).all()) and bool((guard[2] == 5).all())
        assert bool((pool[:2] == 5).all()) and bool((pool[3:] == 5).all()) and bool((pool[2, 1:] == 5).all())


def test_past_32_bits():
    """Tensors of more than 2^32 bytes (2^31 values): the last sequence of a long batch,
    the others zero, gives what it gives alone; so does the last row of a pool."""
    H, d, L, n = 16, 128, 1 << 15, 33  # 33 x 2^15 tokens x 2048 values x 2 bytes = 4.4 GB a tensor
    x = dev(G.make(1, L, H, H, d, d, BF, seed=2, s0=False))
    one = [x[m] for m in G.NAMES]
    o1, S1 = efla.efla_gated_chunk_fwd(*one)
    many = []
    for t in one:
        m = torch.zeros(n, *t.shape[1:], dtype=t.dtype, device="cuda")
        m[-1] = t[0]
        many.append(m)
    o, S = efla.efla_gated_chunk_fwd(*many)
    assert torch.equal(o[-1], o1[0]) and torch.equal(S[-1], S1[0]) and not bool(o[:-1].any())
    del o, S
    cu = torch.arange(0, (n + 1) * L, L, dtype=torch.int32).cuda()
    o, S = efla.efla_gated_chunk_fwd_varlen(*(t.flatten(0, 1) for t in many), cu)
    assert torch.equal(o[-L:], o1[0]) and torch.equal(S[-1], S1[0])
    del o, S
    do = torch.zeros_like(many[2])
    do[-1] = torch.randn(L, H, d, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    want = efla.efla_gated_chunk_bwd(*one, do[-1:].clone())
    got = efla.efla_gated_chunk_bwd(*many, do)
    for name, p, r in zip(GRADS, got, want):
        assert torch.equal(p[-1], r[0]), name
    del got, want, many, do
    P = 4200  # 2^20 bytes a row
    pool = torch.zeros(P, H, d, d, device="cuda")
    st = torch.randn(2, H, d, d, generator=torch.Generator().manual_seed(4)).cuda()
    pool[-2:] = st
    row = [t[0, :2].contiguous() for t in one]
    y1 = efla.efla_gated_step(*row, st)
    y = efla.efla_gated_step(*row, pool, torch.tensor([P - 2, P - 1], dtype=torch.int32).cuda())
    assert torch.equal(y, y1) and torch.equal(pool[-2:], st) and not bool(pool[:-2].any())
