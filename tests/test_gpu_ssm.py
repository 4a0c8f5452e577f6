"""The selective state space scan on the GPU against its 64-bit form: forward, packed
batches with states in a pool, one token a request, and the gradient."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LENGTHS = [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 127, 130, 200, 449]


def dev(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def ins(x):
    return [x[n] for n in ("q", "k", "v", "dt", "a")], dict(d=x["d"], dt_bias=x["bias"])


def check_fwd(x, dtype, L, dk, o, S):
    ro, rs = R.scan_ref(*(None if t is None else t.cpu() for t in R.wide(x)))
    assert o.dtype == dtype and R.rel(o, ro) <= R.tol_o(dtype, L, dk), R.rel(o, ro)
    assert R.rel(S, rs) <= R.tol_s(dtype, L, dk), R.rel(S, rs)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", LENGTHS)
def test_forward_lengths(dtype, L):
    for dk, dv, H, Hk in ((64, 64, 4, 2), (128, 128, 2, 1), (128, 64, 3, 3)):
        x = dev(R.make_scan(2, L, H, Hk, dk, dv, dtype, seed=L, s0=L % 2 == 0))
        a, kw = ins(x)
        o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        check_fwd(x, dtype, L, dk, o, S)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_forward_head_sizes(dtype, dk, dv):
    x = dev(R.make_scan(1, 150, 4, 1, dk, dv, dtype, seed=dk + dv, extras=dk != dv))
    a, kw = ins(x)
    o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    check_fwd(x, dtype, 150, dk, o, S)
    o2, none = efla.efla_ssm_fwd(*a, s0=x["s0"], want_final=False, **kw)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_long_and_many_short_sequences(dtype):
    for B, L, H in ((1, 2500, 2), (700, 5, 8), (40, 70, 16)):
        x = dev(R.make_scan(B, L, H, 1, 64, 64, dtype, seed=B))
        a, kw = ins(x)
        o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        check_fwd(x, dtype, L, 64, o, S)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_parts_of_wider_rows(dtype):
    B, L, H, Hk, dk, dv = 2, 130, 4, 2, 64, 64
    x = dev(R.make_scan(B, L, H, Hk, dk, dv, dtype))
    a, kw = ins(x)
    want, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    # one projection's rows: v, k, q and a stretch that belongs to something else, dt of its own with an odd row
    row = torch.full((B, L, H * dv + 2 * Hk * dk + 8), float("nan"), dtype=dtype, device="cuda")
    v = row[..., :H * dv].unflatten(-1, (H, dv))
    k = row[..., H * dv:H * dv + Hk * dk].unflatten(-1, (Hk, dk))
    q = row[..., H * dv + Hk * dk:H * dv + 2 * Hk * dk].unflatten(-1, (Hk, dk))
    dt = R.in_wider_rows(x["dt"], 2, 3)
    for t, n in ((v, "v"), (k, "k"), (q, "q")):
        t.copy_(x[n])
    out = torch.full((B, L, H * dv + 16), 4.0, dtype=dtype, device="cuda")
    o, S2 = efla.efla_ssm_fwd(q, k, v, dt, x["a"], s0=x["s0"], o=out[..., 16:].unflatten(-1, (H, dv)), **kw)
    assert torch.equal(o, want) and torch.equal(S, S2) and bool((out[..., :16] == 4.0).all())
    d_o = torch.randn(B, L, H, dv, device="cuda").to(dtype)
    want = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
    grow = torch.full_like(row, 4.0)
    gv = grow[..., :H * dv].unflatten(-1, (H, dv))
    gk = grow[..., H * dv:H * dv + Hk * dk].unflatten(-1, (Hk, dk))
    gq = grow[..., H * dv + Hk * dk:H * dv + 2 * Hk * dk].unflatten(-1, (Hk, dk))
    gdt = torch.zeros(B, L, H + 1, dtype=dtype, device="cuda")[..., :H]
    got = efla.efla_ssm_bwd(q, k, v, dt, x["a"], R.in_wider_rows(d_o, 2, 8), s0=x["s0"], dq=gq, dk=gk, dv=gv, ddt=gdt, **kw)
    assert all(torch.equal(p, r) for p, r in zip(got, want)) and bool((grow[..., -8:] == 4.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (16, 32)])
def test_packed_batch(dtype, dk, dv):
    lens = [3, 0, 1, 70, 2, 0, 330, 33, 64, 1, 129, 0]
    N, T, H, Hk = len(lens), sum(lens) + 9, 4, 2
    x = dev(R.make_scan(N + 4, 0, H, Hk, dk, dv, dtype, lead=(T,)))
    a, kw = ins(x)
    plan = efla.efla_pack_plan(torch.tensor(lens, dtype=torch.int32).cuda(), T)
    slots = torch.randperm(N + 4, generator=torch.Generator().manual_seed(1))[:N].to(torch.int32)
    slots[3], slots[7] = -1, N + 4
    results = []
    for alias, order in ((False, None), (True, plan.order)):
        s0 = x["s0"].clone()
        out = s0 if alias else torch.full_like(s0, 7.0)
        o = torch.full((T, H, dv), 3.0, dtype=dtype, device="cuda")
        efla.efla_ssm_fwd_varlen(*a, plan.cu_seqlens, s0=s0, slots=slots.cuda(), order=order, o=o, s_final=out, **kw)
        at, want = 0, x["s0"].clone() if alias else torch.full_like(s0, 7.0)
        for n, slot in zip(lens, slots.tolist()):
            inside = 0 <= slot < N + 4
            part = {m: x[m][None, at:at + n] for m in ("q", "k", "v", "dt")}
            part.update({m: x[m] for m in ("a", "d", "bias")}, s0=x["s0"][slot:slot + 1] if inside else None)
            ro, rs = R.scan_ref(*(None if t is None else t.cpu() for t in R.wide(part)))
            if n:
                assert R.rel(o[None, at:at + n], ro) <= R.tol_o(dtype, n, dk), (n, slot)
            if inside:
                assert R.rel(out[slot:slot + 1], rs) <= R.tol_s(dtype, n, dk), (n, slot)
                want[slot] = out[slot]
            at += n
        assert torch.equal(out, want) and bool((o[at:] == 3.0).all())
        results.append(o)
    assert torch.equal(*results)
    made, none = efla.efla_ssm_fwd_varlen(*a, plan.cu_seqlens, want_final=False, **kw)
    assert none is None and bool((made[at:] == 0).all())
    bad = torch.tensor([5, -3, 1 << 30, 2, 100, -7], dtype=torch.int32).cuda()  # numbers are unspecified, accesses are not
    efla.efla_ssm_fwd_varlen(*a, bad, **kw)
    torch.cuda.synchronize()


def test_no_tokens():
    x = dev(R.make_scan(2, 0, 4, 2, 64, 64, BF))
    a, kw = ins(x)
    o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    assert o.shape == (2, 0, 4, 64) and torch.equal(S, x["s0"])
    _, S = efla.efla_ssm_fwd(*a, **kw)
    assert not S.any()
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    packed = [t[0] for t in a[:4]] + [a[4]]
    _, S = efla.efla_ssm_fwd_varlen(*packed, cu, s0=x["s0"], **kw)
    assert torch.equal(S, x["s0"])
    dsf = torch.randn(2, 4, 64, 64, device="cuda")
    got = efla.efla_ssm_bwd(*a, o, s0=x["s0"], ds_final=dsf, **kw)
    assert torch.equal(got[7], dsf) and not any(bool(t.any()) for t in got[4:7])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,H,Hk,dk,dv", [(1, 4, 2, 64, 64), (5, 16, 4, 128, 128), (3, 3, 1, 16, 32), (130, 16, 1, 128, 64),
                                          (2, 2, 2, 32, 16)])
def test_step_continues_the_forward(dtype, N, H, Hk, dk, dv):
    L = 3
    x = dev(R.make_scan(N, L, H, Hk, dk, dv, dtype))
    a, kw = ins(x)
    st = x["s0"].clone()
    ro, rs = R.scan_ref(*(None if t is None else t.cpu() for t in R.wide(x)))
    for t in range(L):
        o = efla.efla_ssm_step(*(y[:, t] for y in a[:4]), a[4], st, **kw)
        assert R.rel(o, ro[:, t]) <= R.tol32(L, dk) + (2.0 ** -8 if dtype == BF else 0)
    assert R.rel(st, rs) <= R.tol32(L, dk)
    P = N + 3
    pool = torch.randn(P, H, dk, dv, device="cuda")
    slots = torch.randperm(P, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32).cuda()
    if N > 2:
        slots[0], slots[2] = -1, P
    keep, given = pool.clone(), torch.full((N, H, dv), 5.0, dtype=dtype, device="cuda")
    o = efla.efla_ssm_step(*(y[:, 0] for y in a[:4]), a[4], pool, slots=slots, o=given, **kw)
    named = [s for s in slots.tolist() if 0 <= s < P]
    live = [n for n, s in enumerate(slots.tolist()) if 0 <= s < P]
    part = {m: x[m][live, :1] for m in ("q", "k", "v", "dt")}
    part.update({m: x[m] for m in ("a", "d", "bias")}, s0=keep[named])
    ro, rs = R.scan_ref(*(None if t is None else t.cpu() for t in R.wide(part)))
    assert R.rel(o[live], ro[:, 0]) <= R.tol32(1, dk) + (2.0 ** -8 if dtype == BF else 0)
    assert R.rel(pool[named], rs) <= R.tol32(1, dk)
    rest = [i for i in range(P) if i not in named]
    assert torch.equal(pool[rest], keep[rest])
    dead = [n for n in range(N) if n not in live]
    assert bool((o[dead] == 5.0).all())


def check_grads(x, dtype, L, dk, d_o, dsf, got):
    want, scale = R.scan_grads_ref({k: None if v is None else v.cpu() for k, v in x.items()}, d_o.cpu(),
                                   None if dsf is None else dsf.cpu())
    for name, y in zip(R.GRADS, got):
        if want[name] is None:
            assert y is None or name == "ds0"
            continue
        err = R.rel(y, want[name], scale.get(name))
        assert err <= R.tol_grad(dtype, L, dk, name), (name, err, R.tol_grad(dtype, L, dk, name))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [1, 2, 16, 17, 33, 64, 65, 130, 260])
def test_gradient_lengths(dtype, L):
    for dk, dv, H, Hk in ((64, 64, 4, 2), (128, 128, 2, 1), (128, 64, 3, 3)):
        x = dev(R.make_scan(2, L, H, Hk, dk, dv, dtype, seed=L, s0=L % 2 == 0))
        a, kw = ins(x)
        gen = torch.Generator().manual_seed(L)
        d_o = torch.randn(2, L, H, dv, generator=gen).to(dtype).cuda()
        dsf = torch.randn(2, H, dk, dv, generator=gen).cuda() if L % 3 else None
        got = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], ds_final=dsf, **kw)
        check_grads(x, dtype, L, dk, d_o, dsf, got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_gradient_head_sizes(dtype, dk, dv):
    x = dev(R.make_scan(1, 100, 4, 1, dk, dv, dtype, seed=dk + dv, extras=dk != dv))
    a, kw = ins(x)
    d_o = torch.randn(1, 100, 4, dv, generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    got = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
    check_grads(x, dtype, 100, dk, d_o, None, got)
    less = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], want_ds0=False, **kw)
    assert less[7] is None and all(p is None or torch.equal(p, r) for p, r in zip(less, got))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk", [(16, 1), (16, 2), (24, 8), (1, 1), (5, 1)])
def test_gradient_of_shared_heads(dtype, H, Hk):
    x = dev(R.make_scan(2, 90, H, Hk, 64, 64, dtype, seed=H))
    a, kw = ins(x)
    d_o = torch.randn(2, 90, H, 64, generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    got = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
    check_grads(x, dtype, 90, 64, d_o, None, got)
    for _ in range(3):
        again = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
        assert all(torch.equal(p, r) for p, r in zip(got, again))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [16, 64, 100, 300])
@pytest.mark.parametrize("rate", [-16.0, -1.0])
def test_rate_gradient_of_neighbours(dtype, L, rate):
    """Of a head that forgets within a few tokens only near pairs carry da; the errors of the others' products, which
    cancel on each side of a token, may not.  A term has the roundings of two products over 64 and the factors,
    sqrt(64) + 8 half steps; states and their gradients another 3 parts' worth, the same again."""
    x = dev(R.make_scan(2, L, 8, 2, 64, 64, dtype, seed=L, s0=False, steps=(0.05, 0.1)))
    x["q"], x["k"] = x["q"].abs(), x["k"].abs()
    x["a"].fill_(rate)
    a, kw = ins(x)
    d_o = torch.randn(2, L, 8, 64, generator=torch.Generator().manual_seed(L)).to(dtype).cuda()
    da = efla.efla_ssm_bwd(*a, d_o, **kw)[4].double().cpu()
    want, scale = R.rate_gradient_ref({n: None if t is None else t.cpu() for n, t in x.items()}, d_o.cpu())
    assert bool(((da - want).abs() <= 32 * 2.0 ** -24 * scale).all()), ((da - want) / scale * 2.0 ** 24).tolist()


def test_gradient_against_differences():
    x = R.make_scan(1, 40, 2, 1, 16, 16, F32)
    gen = torch.Generator().manual_seed(3)
    d_o, dsf = torch.randn(1, 40, 2, 16, generator=gen), torch.randn(1, 2, 16, 16, generator=gen)
    a, kw = ins(dev(x))
    got = efla.efla_ssm_bwd(*a, d_o.cuda(), s0=x["s0"].cuda(), ds_final=dsf.cuda(), **kw)
    for name, g in zip(R.NAMES, got):
        way = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        loss = []
        for sign in (1, -1):
            y = {n: x[n].double() + (sign * 1e-5 * way if n == name else 0) for n in x}
            o, S = R.scan_ref(*(y[n] for n in R.NAMES))
            loss.append(float((o * d_o).sum() + (S * dsf).sum()))
        slope, along = (loss[0] - loss[1]) / 2e-5, float((g.double().cpu() * way).sum())
        assert abs(slope - along) <= 1e-5 * float(g.double().norm().cpu() * way.norm()), name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_extreme_steps(dtype):
    """Steps of zero (dt = -inf) leave the state, large ones replace it, and neither makes a NaN; slow and fast heads."""
    for L in (40, 150):
        x = R.make_scan(1, L, 4, 2, 64, 64, dtype, steps=(1e-4, 3.0))
        x["dt"][:, 5:9] = float("-inf")
        x["dt"][:, 20] = 200.0
        x["dt"][:, L - 3, :2] = 60.0
        x["a"] = torch.tensor([-1e-4, -1.0, -16.0, 0.0])
        x = dev(x)
        a, kw = ins(x)
        o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        check_fwd(x, dtype, L, 64, o, S)
        d_o = torch.randn(1, L, 4, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        got = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
        assert all(bool(t.isfinite().all()) for t in got)
        check_grads(x, dtype, L, 64, d_o, None, got)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_nan_stays_in_its_sequence(dtype):
    lens = [70, 200, 33, 64]
    T = sum(lens)
    x = dev(R.make_scan(4, 0, 4, 2, 64, 64, dtype, lead=(T,)))
    a, kw = ins(x)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    want, S = efla.efla_ssm_fwd_varlen(*a, cu, s0=x["s0"], **kw)
    for name in ("q", "k", "v", "dt"):
        y = dict(x)
        y[name] = x[name].clone()
        y[name][70 + 130] = float("nan")  # token 130 of the second sequence
        b, _ = ins(y)
        o, S2 = efla.efla_ssm_fwd_varlen(*b, cu, s0=x["s0"], **kw)
        same = [0, 2, 3]
        assert torch.equal(S2[same], S[same])
        assert torch.equal(o[:70 + 128], want[:70 + 128]) and torch.equal(o[270:], want[270:])
        assert bool(o[200].isnan().any())


def test_rows_beyond_32_bit_offsets():
    """Token rows 2^24 - 8 elements apart: the last of 300 lies past 2^32 elements of its tensor."""
    H, d, L, row = 2, 64, 300, 2 ** 24 - 8
    x = dev(R.make_scan(1, L, H, 1, d, d, BF))
    a, kw = ins(x)
    want, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    big = torch.empty((L - 1) * row + 4 * H * d, dtype=BF, device="cuda")

    def place(t, at):
        n = t[0, 0].numel()
        view = big.as_strided((1, L, *t.shape[2:]), (L * row, row, *([t.shape[3], 1] if t.dim() == 4 else [1])), at)
        view.copy_(t)
        return view, at + -(-n // 8) * 8

    v, at = place(x["v"], 0)
    k, at = place(x["k"], at)
    q, at = place(x["q"], at)
    dt, at = place(x["dt"], at)
    o, S2 = efla.efla_ssm_fwd(q, k, v, dt, x["a"], s0=x["s0"], **kw)
    assert torch.equal(o, want) and torch.equal(S, S2)
    d_o = torch.randn(1, L, H, d, device="cuda").to(BF)
    want = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
    got = efla.efla_ssm_bwd(q, k, v, dt, x["a"], d_o, s0=x["s0"], **kw)
    assert all(torch.equal(p, r) for p, r in zip(got, want))
    w = R.make_conv(1, 0, 4 * H * d - 256, 4, BF)
    xs = big.as_strided((1, L, 256), (L * row, row, 1))
    y, _ = efla.efla_conv_fwd(xs, w["w"].cuda()[:256], w["bias"].cuda()[:256])
    y2, _ = efla.efla_conv_fwd(xs.contiguous(), w["w"].cuda()[:256], w["bias"].cuda()[:256])
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_another_stream_and_a_captured_graph(dtype):
    x = dev(R.make_scan(2, 200, 4, 2, 64, 64, dtype))
    a, kw = ins(x)
    d_o = torch.randn(2, 200, 4, 64, device="cuda").to(dtype)
    o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    g = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, S2 = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        g2 = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(p, r) for p, r in zip(g, g2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, S3 = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        g3 = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
    for i in range(3):
        x["v"].copy_(torch.randn(2, 200, 4, 64, device="cuda").to(dtype))
        graph.replay()
        torch.cuda.synchronize()
        o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        g = efla.efla_ssm_bwd(*a, d_o, s0=x["s0"], **kw)
        assert torch.equal(o, o3) and torch.equal(S, S3) and all(torch.equal(p, r) for p, r in zip(g, g3)), i


def layer(x, w, cu=None, step=None, train=None):
    """A layer's convolution and scan on the rows of one projection [.., v | k | q | dt]."""
    H, Hk, dk, dv = w["sizes"]
    D, nv, nk = w["conv"].shape[0], H * dv, Hk * dk

    def parts(y):
        return (y[..., nv + nk:D].unflatten(-1, (Hk, dk)), y[..., nv:nv + nk].unflatten(-1, (Hk, dk)),
                y[..., :nv].unflatten(-1, (H, dv)))

    kw = dict(d=w["d"], dt_bias=w["bias"])
    inp, dt = x[..., :D], x[..., D:]
    if step is not None:
        conv, state, slots = step
        y = efla.efla_conv_step(inp, w["conv"], conv, w["cbias"], slots)
        return efla.efla_ssm_step(*parts(y), dt, w["a"], state, slots=slots, **kw)
    if cu is not None:
        offsets, slots, conv, state = cu
        y, _ = efla.efla_conv_fwd_varlen(inp, w["conv"], offsets, w["cbias"], conv, slots, s_final=conv)
        o, _ = efla.efla_ssm_fwd_varlen(*parts(y), dt, w["a"], offsets, s0=state, slots=slots, s_final=state, **kw)
        return o
    y, cf = efla.efla_conv_fwd(inp, w["conv"], w["cbias"])
    o, S = efla.efla_ssm_fwd(*parts(y), dt, w["a"], **kw)
    if train is None:
        return o, cf, S
    gy, gx = torch.empty_like(y), torch.empty_like(x)
    gq, gk, gv = parts(gy)
    rest = efla.efla_ssm_bwd(*parts(y), dt, w["a"], train, dq=gq, dk=gk, dv=gv, ddt=gx[..., D:], want_ds0=False, **kw)
    _, dw, db, _ = efla.efla_conv_bwd(inp, w["conv"], gy, w["cbias"], dx=gx[..., :D], want_ds0=False)
    return o, gx, dw, db, *rest[4:7]


def make_layer(dtype, H=4, Hk=2, dk=64, dv=64):
    gen = torch.Generator().manual_seed(0)
    x = R.make_scan(1, 1, H, Hk, dk, dv, dtype)
    D = H * dv + 2 * Hk * dk
    return {"sizes": (H, Hk, dk, dv), "conv": (0.5 * torch.randn(D, 4, generator=gen)).to(dtype).cuda(),
            "cbias": (0.1 * torch.randn(D, generator=gen)).to(dtype).cuda(), "a": x["a"].cuda(), "d": x["d"].cuda(),
            "bias": x["bias"].cuda()}


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompts_forks_and_tokens_of_a_layer(dtype):
    """A serving run: prompts prefilled into pools, one forked, the batch decoded, a request ended, the pools compacted
    and the rest decoded; each continuation equals its whole sequence run at once."""
    w = make_layer(dtype)
    H, Hk, dk, dv = w["sizes"]
    D, P = w["conv"].shape[0], 8
    gen = torch.Generator().manual_seed(4)
    lens = [37, 5, 90]
    prompt = torch.randn(sum(lens), D + H, generator=gen).to(dtype).cuda()
    conv = torch.zeros(P, 3, D, dtype=dtype, device="cuda")
    state = torch.zeros(P, H, dk, dv, device="cuda")
    slots = torch.tensor([6, 2, 7], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 37, 42, 132], dtype=torch.int32, device="cuda")
    layer(prompt, w, cu=(cu, slots, conv, state))
    i32 = dict(dtype=torch.int32, device="cuda")
    efla.efla_pool_copy([state, conv], torch.tensor([6, 6], **i32), torch.tensor([0, 4], **i32))  # two more of request 0
    slots = torch.tensor([6, 2, 7, 0, 4, -1], **i32)
    owner = [0, 1, 2, 0, 0]
    seqs = [prompt[int(cu[i]):int(cu[i + 1])] for i in owner]
    for turn in range(4):
        if turn == 2:  # request 1 ends; the five others' rows move to the front
            slots = torch.tensor([6, 7, 0, 4, -1, -1], **i32)
            seqs = [seqs[0], seqs[2], seqs[3], seqs[4]]
            slots, live = efla.efla_pool_compact([state, conv], slots)
            assert int(live) == 4 and sorted(slots.tolist()[:4]) == [0, 1, 2, 3] and slots.tolist()[4:] == [-1, -1]
        x = torch.randn(6, D + H, generator=gen).to(dtype).cuda()
        o = layer(x, w, step=(conv, state, slots))
        seqs = [torch.cat([s, x[i:i + 1]]) for i, s in enumerate(seqs)]
        for i, s in enumerate(seqs):
            want, cf, S = layer(s[None], w)
            assert R.rel(o[i], want[0, -1]) <= 2 * R.tol_o(dtype, len(s), dk) + R.tol_conv(dtype)
            row = int(slots[i])
            assert torch.equal(conv[row], cf[0])
            # the prompt's q, k and v are the same rounded values in both runs
            assert R.rel(state[row], S[0]) <= 2 * R.tol_s(dtype, len(s), dk)


def test_training_step_of_a_layer():
    w = make_layer(F32, H=2, Hk=1, dk=16, dv=16)
    H, Hk, dk, dv = w["sizes"]
    D = w["conv"].shape[0]
    gen = torch.Generator().manual_seed(7)
    x, d_o = torch.randn(2, 75, D + H, generator=gen), torch.randn(2, 75, H, dv, generator=gen)
    got = layer(x.cuda(), w, train=d_o.cuda())
    leaves = [t.double().cpu().requires_grad_() for t in (x, w["conv"], w["cbias"], w["a"], w["d"], w["bias"])]
    xx, cw, cb, a, d, bias = leaves
    y, _ = R.conv_ref(xx[..., :D], cw, cb)
    nv, nk = H * dv, Hk * dk
    o, _ = R.scan_ref(y[..., nv + nk:].unflatten(-1, (Hk, dk)), y[..., nv:nv + nk].unflatten(-1, (Hk, dk)),
                      y[..., :nv].unflatten(-1, (H, dv)), xx[..., D:], a, d, bias)
    want = torch.autograd.grad((o * d_o).sum(), leaves)
    assert R.rel(got[0], o) <= R.tol32(75, dk)
    for g, r in zip(got[1:], want):
        assert R.rel(g, r) <= R.tol32(75, dk, "grad")
