"""The gated delta rule on the GPU against the token-by-token form in 64 bits
(tests/_gated.py holds it and the tolerances' derivation)."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _gated as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def dev(x):
    return {n: (None if t is None else t.cuda()) for n, t in x.items()}


def ids(p):
    return "-".join(str(x).replace("torch.", "") for x in p)


# ------------------------------------------------------------------ decode
STEP = [(1, 1, 1, 16, 16, F32, "exact"), (1, 16, 16, 128, 128, BF, "euler"), (3, 4, 2, 32, 64, F32, "euler"),
        (5, 8, 2, 64, 128, BF, "exact"), (40, 16, 16, 128, 128, BF, "exact"), (2, 6, 3, 128, 16, F32, "exact"),
        (33, 16, 4, 16, 128, BF, "euler"), (70, 8, 8, 64, 64, F32, "exact")]


@pytest.mark.parametrize("p", STEP, ids=ids)
def test_step(p):
    N, H, Hk, dk, dv, dt, rule = p
    x = G.make(N, 3, H, Hk, dk, dv, dt, seed=N + dk)
    d = dev(x)
    state = d["s0"].clone()
    outs = [efla.efla_gated_step(*(d[n][:, t].contiguous() for n in G.NAMES), state, rule=rule) for t in range(3)]
    o, S = G.forward_ref(*G.wide(x), x["s0"].double(), rule)
    assert G.rel(torch.stack(outs, 1), o) <= (G.tol32(3, dk) if dt == F32 else 2.0 ** -8 + G.tol32(3, dk))
    assert G.rel(state, S) <= G.tol32(3, dk)  # the step is float32 arithmetic whatever the inputs' type


def test_step_pool_rows_and_skipped_rows():
    N, P, H, dk, dv = 7, 11, 4, 64, 32
    x = dev(G.make(N, 1, H, 2, dk, dv, BF, seed=3, s0=False))
    pool = torch.randn(P, H, dk, dv, generator=torch.Generator().manual_seed(4)).cuda()
    slots = torch.tensor([9, -1, 0, 10, 2 ** 30, 5, -(2 ** 31)], dtype=torch.int32).cuda()
    live = [0, 2, 3, 5]
    before = pool.clone()
    o = torch.full((N, H, dv), 7.0, dtype=BF).cuda()
    a = [x[n][:, 0].contiguous() for n in G.NAMES]
    assert efla.efla_gated_step(*a, pool, slots=slots, o=o) is o
    want = before[slots[live].long()].clone()
    o2 = efla.efla_gated_step(*(t[live].contiguous() for t in a), want)
    assert torch.equal(o[live], o2) and bool((o[[1, 4, 6]] == 7.0).all())
    assert torch.equal(pool[slots[live].long()], want)
    rest = [i for i in range(P) if i not in slots[live].tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_step_reset_and_growth():
    """g = -inf forgets the state, g = 0 keeps it, a positive g grows it."""
    x = G.make(3, 1, 2, 2, 32, 32, F32, seed=5)
    x["g"] = torch.tensor([float("-inf"), 0.0, 1.5]).reshape(3, 1, 1).expand(3, 1, 2).contiguous()
    d = dev(x)
    S = d["s0"].clone()
    efla.efla_gated_step(*(d[n][:, 0].contiguous() for n in G.NAMES), S)
    _, want = G.forward_ref(*G.wide(x), x["s0"].double())
    assert G.rel(S, want) <= G.tol32(1, 32)


# ----------------------------------------------------------------- forward
FWD = [(1, 1, 1, 1, 16, 16, 64, F32, "exact"), (2, 17, 4, 2, 32, 16, 16, F32, "euler"),
       (1, 64, 2, 2, 64, 64, 64, F32, "exact"), (2, 129, 4, 1, 128, 32, 32, F32, "euler"),
       (1, 1, 2, 2, 128, 128, 64, BF, "euler"), (2, 63, 4, 4, 64, 64, 64, BF, "exact"),
       (1, 64, 2, 1, 128, 128, 64, BF, "exact"), (1, 65, 8, 2, 128, 64, 64, BF, "euler"),
       (3, 200, 4, 2, 64, 128, 64, BF, "euler"), (1, 321, 2, 2, 128, 128, 64, BF, "exact"),
       (2, 100, 2, 2, 32, 32, 64, BF, "exact"), (1, 90, 3, 3, 128, 16, 64, BF, "euler"),
       (1, 150, 4, 4, 64, 64, 32, BF, "exact"), (8, 130, 8, 8, 128, 128, 64, BF, "euler")]


@pytest.mark.parametrize("p", FWD, ids=ids)
def test_forward(p):
    B, L, H, Hk, dk, dv, C, dt, rule = p
    x = G.make(B, L, H, Hk, dk, dv, dt, seed=L)
    d = dev(x)
    o, S = efla.efla_gated_chunk_fwd(*(d[n] for n in G.NAMES), d["s0"], chunk=C, rule=rule)
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double(), rule)
    assert G.rel(o, wo) <= G.tol_o(dt, L, dk)
    assert G.rel(S, wS) <= G.tol_s(dt, L, dk)


def test_forward_no_state_no_final_and_empty():
    x = G.make(1, 70, 4, 4, 64, 64, BF, seed=1, s0=False)
    d = dev(x)
    a = [d[n] for n in G.NAMES]
    o, S = efla.efla_gated_chunk_fwd(*a, want_final=False)
    assert S is None
    assert G.rel(o, G.forward_ref(*G.wide(x))[0]) <= G.tol_o(BF, 70, 64)
    s0 = torch.randn(1, 4, 64, 64).cuda()
    o, S = efla.efla_gated_chunk_fwd(*(t[:, :0].contiguous() for t in a), s0)
    assert o.shape[1] == 0 and torch.equal(S, s0)


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
def test_forward_without_decay_is_the_delta_rule(dt):
    x = dev(G.make(2, 150, 4, 4, 64, 64, dt, seed=8))
    x["g"].zero_()
    o, S = efla.efla_gated_chunk_fwd(*(x[n] for n in G.NAMES), x["s0"])
    o2, S2 = efla.efla_chunk_fwd(x["q"], x["k"], x["v"], x["beta"], x["s0"])
    assert G.rel(o, o2) <= (2e-5 if dt == F32 else 2e-2) and G.rel(S, S2) <= (2e-5 if dt == F32 else 1e-2)


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
def test_forward_extreme_gates(dt):
    """Resets (-inf, the type's lowest), no decay, growth and strong decay in one sequence."""
    L = 200
    x = G.make(1, L, 2, 2, 64, 64, dt, seed=6, decay=2.0)
    g = x["g"]
    g[:, 5], g[:, 70], g[:, 71] = float("-inf"), torch.finfo(F32).min, float("-inf")
    g[:, 100:110], g[:, 110:120] = 0.0, 0.05
    g[:, 199] = -300.0
    d = dev(x)
    o, S = efla.efla_gated_chunk_fwd(*(d[n] for n in G.NAMES), d["s0"])
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double())
    # sums of gates reach 300 in a chunk: their float32 differences are off by 300 * 2^-24 each, twice
    extra = 2 * 300 * 2.0 ** -23
    assert bool(torch.isfinite(o).all()) and G.rel(o, wo) <= G.tol_o(dt, L, 64) + extra
    assert G.rel(S, wS) <= G.tol_s(dt, L, 64) + extra


def test_forward_nan_stays_in_its_sequence():
    x = dev(G.make(3, 80, 2, 2, 64, 64, BF, seed=9))
    clean, _ = efla.efla_gated_chunk_fwd(*(x[n] for n in G.NAMES), x["s0"])
    x["v"][1, 40, 0, 3] = float("nan")
    o, S = efla.efla_gated_chunk_fwd(*(x[n] for n in G.NAMES), x["s0"])
    assert torch.equal(o[0], clean[0]) and torch.equal(o[2], clean[2]) and torch.equal(o[1, :, 1], clean[1, :, 1])
    assert bool(S[1, 0].isnan().any()) and bool(S[0].isfinite().all())


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
def test_forward_then_steps_is_one_sequence(dt):
    """A prompt through the chunked pass, then tokens one by one, equals the whole sequence."""
    x = G.make(2, 133, 4, 2, 64, 64, dt, seed=10)
    d = dev(x)
    _, S = efla.efla_gated_chunk_fwd(*(d[n][:, :130].contiguous() for n in G.NAMES), d["s0"], rule="euler")
    outs = [efla.efla_gated_step(*(d[n][:, t].contiguous() for n in G.NAMES), S, rule="euler") for t in range(130, 133)]
    wo, wS = G.forward_ref(*G.wide(x), x["s0"].double(), "euler")
    assert G.rel(S, wS) <= G.tol_s(dt, 133, 64)
    assert G.rel(torch.stack(outs, 1), wo[:, 130:]) <= G.tol_o(dt, 133, 64)


# ------------------------------------------------------------------ packed
VAR = [([1], 4, 4, 64, 64, F32), ([5, 0, 64, 1, 63, 65], 4, 2, 64, 64, BF), ([0, 0, 130], 2, 2, 128, 128, BF),
       ([16, 17, 200, 3], 4, 1, 32, 16, F32), ([7] * 20, 2, 2, 128, 64, BF), ([300, 1, 129], 8, 8, 64, 128, BF)]


@pytest.mark.parametrize("p", VAR, ids=lambda p: ids((len(p[0]),) + p[1:]))
@pytest.mark.parametrize("pooled", [False, True])
def test_varlen(p, pooled):
    lens, H, Hk, dk, dv, dt = p
    N, T = len(lens), sum(lens) + 9  # 4 rows before and 5 behind the sequences
    x = G.make(N, 0, H, Hk, dk, dv, dt, seed=T, lead=(T,))
    d = dev(x)
    cu = torch.tensor([4] + [4 + sum(lens[:i + 1]) for i in range(N)], dtype=torch.int32).cuda()
    kw = {}
    if pooled:
        perm = torch.randperm(N + 2, generator=torch.Generator().manual_seed(1))[:N].to(torch.int32)
        pool = torch.randn(N + 2, H, dk, dv, generator=torch.Generator().manual_seed(2)).cuda()
        s0 = pool[perm.long().cuda()].clone()
        before = pool.clone()
        kw = dict(slots=perm.cuda(), s_final=pool)  # in place
        start = pool
    else:
        s0 = start = d["s0"]
    o = torch.full((T, H, dv), 5.0, dtype=dt).cuda()
    got, S = efla.efla_gated_chunk_fwd_varlen(*(d[n] for n in G.NAMES), cu, start, o=o, rule="euler", **kw)
    assert got is o and bool((o[:4] == 5.0).all()) and bool((o[T - 5:] == 5.0).all())
    for i, n in enumerate(lens):
        a = 4 + sum(lens[:i])
        wo, wS = G.forward_ref(*(t[None, a:a + n] for t in G.wide(x)), s0[i:i + 1].double().cpu(), "euler")
        if n:
            assert G.rel(o[a:a + n], wo[0]) <= G.tol_o(dt, n, dk)
        Si = S[int(perm[i])] if pooled else S[i]
        assert G.rel(Si, wS[0]) <= G.tol_s(dt, n, dk)
    if pooled:
        rest = [i for i in range(N + 2) if i not in perm.tolist()]
        assert torch.equal(pool[rest], before[rest])


def test_varlen_slots_without_a_row():
    """An entry outside the pool: from zero, and no final state."""
    lens, H, d_ = [40, 70], 2, 64
    x = dev(G.make(2, 0, H, H, d_, d_, BF, seed=2, lead=(110,)))
    cu = torch.tensor([0, 40, 110], dtype=torch.int32).cuda()
    a = [x[n] for n in G.NAMES]
    pool = torch.randn(3, H, d_, d_).cuda()
    before = pool.clone()
    o, _ = efla.efla_gated_chunk_fwd_varlen(*a, cu, pool, slots=torch.tensor([-1, 3], dtype=torch.int32).cuda(), s_final=pool)
    o2, _ = efla.efla_gated_chunk_fwd_varlen(*a, cu, want_final=False)
    assert torch.equal(o, o2) and torch.equal(pool, before)


# ---------------------------------------------------------------- backward
BWD = [(1, 1, 1, 1, 16, 16, 16, F32, "exact", True), (2, 17, 4, 2, 32, 16, 16, F32, "euler", True),
       (1, 64, 2, 2, 64, 64, 64, F32, "exact", False), (1, 130, 4, 1, 128, 32, 32, F32, "exact", True),
       (1, 65, 2, 2, 128, 128, 64, F32, "euler", True), (1, 1, 2, 2, 64, 64, 64, BF, "euler", True),
       (2, 63, 4, 4, 64, 64, 64, BF, "exact", True), (1, 129, 4, 2, 128, 128, 64, BF, "euler", True),
       (1, 200, 8, 2, 64, 128, 64, BF, "exact", False), (2, 257, 2, 2, 128, 64, 64, BF, "exact", True),
       (1, 70, 2, 2, 32, 32, 32, BF, "euler", True), (1, 90, 2, 1, 128, 16, 64, BF, "exact", True)]
GRADS = ("dq", "dk", "dv", "dbeta", "dg", "ds0")


def grads_ref(x, do, dsf, rule):
    leaves = [t.requires_grad_() for t in G.wide(x)]
    s0 = x["s0"].double().requires_grad_()
    o, S = G.forward_ref(*leaves, s0, rule)
    loss = (o * do.double()).sum() + (0 if dsf is None else (S * dsf.double()).sum())
    return torch.autograd.grad(loss, [*leaves, s0])


@pytest.mark.parametrize("p", BWD, ids=ids)
def test_backward(p):
    B, L, H, Hk, dk, dv, C, dt, rule, final = p
    x = G.make(B, L, H, Hk, dk, dv, dt, seed=L + 1)
    gen = torch.Generator().manual_seed(77)
    do = torch.randn(B, L, H, dv, generator=gen).to(dt)
    dsf = torch.randn(B, H, dk, dv, generator=gen) if final else None
    d = dev(x)
    got = efla.efla_gated_chunk_bwd(*(d[n] for n in G.NAMES), do.cuda(), d["s0"], None if dsf is None else dsf.cuda(),
                                    chunk=C, rule=rule)
    want = grads_ref(x, do, dsf, rule)
    for name, a, b in zip(GRADS, got, want):
        assert a.dtype == (F32 if name == "ds0" else dt)
        assert G.rel(a, b) <= G.tol_grad(dt, L, dk), name


@pytest.mark.parametrize("rule", ["exact", "euler"])
def test_backward_against_differences(rule):
    """Directional derivatives of the 64-bit forward by central differences."""
    B, L, H, Hk, dk, dv = 1, 70, 2, 1, 32, 32
    x = G.make(B, L, H, Hk, dk, dv, F32, seed=12)
    do = torch.randn(B, L, H, dv, generator=torch.Generator().manual_seed(1))
    d = dev(x)
    got = efla.efla_gated_chunk_bwd(*(d[n] for n in G.NAMES), do.cuda(), d["s0"], rule=rule)
    base = [*G.wide(x), x["s0"].double()]
    for i, (name, gr) in enumerate(zip(GRADS, got)):
        way = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        # central difference: truncation eps^2, rounding 2^-53 / eps; at 1e-5 both are far below 1e-4
        f = []
        for s in (1e-5, -1e-5):
            y = list(base)
            y[i] = y[i] + s * way
            f.append(float((G.forward_ref(*y, rule=rule)[0] * do.double()).sum()))
        want = (f[0] - f[1]) / 2e-5
        have = float((gr.double().cpu() * way).sum())
        scale = float(gr.double().norm().cpu() * way.norm()) / way.numel() ** 0.5
        assert abs(have - want) <= 1e-4 * max(scale, abs(want)), name


def test_backward_empty_sequence_passes_the_state_gradient():
    x = dev(G.make(1, 0, 2, 2, 64, 64, BF, seed=1))
    dsf = torch.randn(1, 2, 64, 64).cuda()
    got = efla.efla_gated_chunk_bwd(*(x[n] for n in G.NAMES), torch.empty_like(x["v"]), x["s0"], dsf)
    assert torch.equal(got[5], dsf)


def test_same_call_same_bits():
    x = dev(G.make(2, 300, 4, 2, 128, 128, BF, seed=3))
    do = torch.randn(2, 300, 4, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    a = [x[n] for n in G.NAMES]
    for f in (lambda: efla.efla_gated_chunk_fwd(*a, x["s0"]), lambda: efla.efla_gated_chunk_bwd(*a, do, x["s0"])):
        one = f()
        for _ in range(3):
            assert all(torch.equal(p, q) for p, q in zip(one, f()))


# -------------------------------------------------------------------- plan
PLAN = [([], 5), ([0], 0), ([3], 3), ([0, 0, 0], 7), ([5, 0, 64, 1, 63, 65], 250), ([100, 200], 150), ([-4, 10, 2 ** 31 - 1, 3], 40),
        ([1] * 300, 300), (list(range(100)), 5000)]


@pytest.mark.parametrize("lens,T", PLAN, ids=lambda v: str(len(v)) if isinstance(v, list) else str(v))
@pytest.mark.parametrize("chunk", [16, 64])
def test_plan(lens, T, chunk):
    starts = [(7 * i) % 50 for i in range(len(lens))]
    p = efla.efla_pack_plan(torch.tensor(lens, dtype=torch.int32).cuda(), T, torch.tensor(starts, dtype=torch.int32).cuda(), chunk)
    cu, order, seq, pos = G.plan_ref(lens, T, starts, chunk)
    assert p.cu_seqlens.tolist() == cu and p.order.tolist() == order
    assert p.token_seq.tolist() == seq and p.token_pos.tolist() == pos


@pytest.mark.parametrize("n", [4096, 4097, 9000])
def test_plan_many(n):
    gen = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 9, (n,), generator=gen, dtype=torch.int32)
    T = int(lens.sum()) + 3
    p = efla.efla_pack_plan(lens.cuda(), T)
    cu, order, seq, pos = G.plan_ref(lens.tolist(), T)
    assert p.cu_seqlens.tolist() == cu and p.order.tolist() == order
    assert p.token_seq.tolist() == seq and p.token_pos.tolist() == pos


# ------------------------------------------------- the operators as they are used together
def test_serving_run():
    """Lengths on the GPU -> plan -> packed prompts into a state pool -> decode steps from the pool."""
    lens, H, Hk, dk, dv = [70, 0, 3, 130], 4, 2, 64, 64
    N, T, steps = len(lens), sum(lens), 2
    full = [G.make(1, n + steps, H, Hk, dk, dv, BF, seed=40 + i, s0=False) for i, n in enumerate(lens)]
    pool = torch.zeros(6, H, dk, dv).cuda()
    slots = torch.tensor([4, 2, 0, 5], dtype=torch.int32).cuda()
    plan = efla.efla_pack_plan(torch.tensor(lens, dtype=torch.int32).cuda(), T)
    packed = [torch.cat([f[n][0, :m] for f, m in zip(full, lens)]).cuda() for n in G.NAMES]
    o, _ = efla.efla_gated_chunk_fwd_varlen(*packed, plan.cu_seqlens, pool, slots=slots, order=plan.order, s_final=pool)
    outs = [[o[plan.token_seq == i]] for i in range(N)]
    for t in range(steps):
        tok = [torch.cat([f[n][:, m + t] for f, m in zip(full, lens)]).contiguous().cuda() for n in G.NAMES]
        y = efla.efla_gated_step(*tok, pool, slots=slots)
        for i in range(N):
            outs[i].append(y[i:i + 1])
    for i, f in enumerate(full):
        wo, wS = G.forward_ref(*G.wide(f))
        L = lens[i] + steps
        assert G.rel(torch.cat(outs[i]), wo[0]) <= G.tol_o(BF, L, dk)
        assert G.rel(pool[int(slots[i])], wS[0]) <= G.tol_s(BF, L, dk)


def test_training_step_through_autograd():
    """The forward and backward entry points as one differentiable layer with torch around it."""
    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, beta, g):
            ctx.save_for_backward(q, k, v, beta, g)
            return efla.efla_gated_chunk_fwd(q, k, v, beta, g, want_final=False, rule="euler")[0]

        @staticmethod
        def backward(ctx, do):
            gr = efla.efla_gated_chunk_bwd(*ctx.saved_tensors, do.contiguous(), rule="euler", want_ds0=False)
            return (*gr[:4], gr[4].float())

    x = G.make(1, 100, 2, 1, 32, 32, F32, seed=21, s0=False)
    lv = [x[n].cuda().requires_grad_() for n in G.NAMES]
    ((Layer.apply(*lv) ** 2).sum() * 0.5).backward()
    ref = [t.requires_grad_() for t in G.wide(x)]
    o, _ = G.forward_ref(*ref, rule="euler")
    ((o ** 2).sum() * 0.5).backward()
    for a, b in zip(lv, ref):
        assert G.rel(a.grad, b.grad) <= 2 * G.tol_grad(F32, 100, 32)


def _graph(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = fn()
    return gr, out


def test_captured_and_replayed():
    """Every entry point in a captured graph, replayed on new inputs with eager work between the replays."""
    H, dk, dv = 4, 128, 128
    x = dev(G.make(2, 150, H, 2, dk, dv, BF, seed=1))
    do = torch.randn(2, 150, H, dv, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    a = [x[n] for n in G.NAMES]
    lens = torch.tensor([100, 50], dtype=torch.int32).cuda()
    packed = [t[0] for t in a]

    def run():
        p = efla.efla_pack_plan(lens, 150)
        o, S = efla.efla_gated_chunk_fwd(*a, x["s0"])
        o2, S2 = efla.efla_gated_chunk_fwd_varlen(*packed, p.cu_seqlens, x["s0"], order=p.order)
        y = efla.efla_gated_step(*(t[:, 0].contiguous() for t in a), S)
        return (*p, o, S, o2, S2, y, *efla.efla_gated_chunk_bwd(*a, do, x["s0"]))

    gr, out = _graph(run)
    for i in range(3):
        x["v"].copy_(torch.randn(2, 150, H, dv, generator=torch.Generator().manual_seed(i)))
        lens.copy_(torch.tensor([30 + i, 120 - i], dtype=torch.int32))
        gr.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, run()):
            assert torch.equal(p, q)
        torch.cuda.synchronize()


def test_two_streams_at_once():
    x = dev(G.make(2, 200, 4, 4, 128, 128, BF, seed=2))
    a = [x[n] for n in G.NAMES]
    do = torch.randn(2, 200, 4, 128, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    want = efla.efla_gated_chunk_fwd(*a, x["s0"]) + efla.efla_gated_chunk_bwd(*a, do, x["s0"])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(efla.efla_gated_chunk_fwd(*a, x["s0"]) + efla.efla_gated_chunk_bwd(*a, do, x["s0"]))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(p, q) for p, q in zip(r, want))
