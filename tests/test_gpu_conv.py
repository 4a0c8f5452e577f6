"""The short causal convolution on the GPU against its 64-bit form: forward, packed
batches with states in a pool, one token a request, and the gradient."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def dev(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def wide(t):
    return None if t is None else t.double().cpu()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,L,D", [(1, 1, 8), (2, 2, 24), (1, 3, 1), (3, 7, 513), (2, 64, 512), (1, 257, 520), (2, 300, 37),
                                   (1, 1030, 1000)])
def test_forward(dtype, W, B, L, D):
    for s0, bias, act in ((True, True, "silu"), (False, False, None)):
        x = dev(R.make_conv(B, L, D, W, dtype, seed=L + W, s0=s0, bias=bias))
        y, fin = efla.efla_conv_fwd(x["x"], x["w"], x["bias"], x["s0"], activation=act)
        ry, rf = R.conv_ref(*(wide(x[n]) for n in ("x", "w", "bias", "s0")), silu=act == "silu")
        assert y.dtype == dtype and R.rel(y, ry) <= R.tol_conv(dtype)
        assert torch.equal(fin.cpu().double(), rf)


@pytest.mark.parametrize("D,extra", [(64, 8), (64, 3), (72, 40), (40, 0)])
def test_rows_of_a_wider_tensor(D, extra):
    x = R.make_conv(2, 90, D, 4, BF)
    want, fin = efla.efla_conv_fwd(*(x[n].cuda() for n in ("x", "w", "bias", "s0")))
    for shift in (0, 1):  # a row that starts on 16 bytes, and one that does not
        rows = torch.full((2, 90, shift + D + extra), float("nan"), dtype=BF, device="cuda")
        view, out = rows[..., shift:shift + D], torch.zeros_like(rows)[..., shift:shift + D]
        view.copy_(x["x"])
        y, f = efla.efla_conv_fwd(view, *(x[n].cuda() for n in ("w", "bias", "s0")), y=out)
        assert y is out and torch.equal(y, want) and torch.equal(f, fin)


def test_the_final_state_in_place_of_the_first():
    for L in (0, 1, 2, 3, 50):
        x = dev(R.make_conv(2, L, 72, 4, BF, seed=L))
        y, fin = efla.efla_conv_fwd(x["x"], x["w"], x["bias"], x["s0"])
        st = x["s0"].clone()
        y2, f2 = efla.efla_conv_fwd(x["x"], x["w"], x["bias"], st, s_final=st)
        assert f2 is st and torch.equal(y, y2) and torch.equal(fin, st)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 1030])
def test_packed_batch(dtype, D):
    lens = [3, 0, 1, 70, 2, 0, 130, 33, 1, 1, 64, 0]
    N, T, W = len(lens), sum(lens) + 11, 4
    x = dev(R.make_conv(N + 4, 0, D, W, dtype, lead=(T,)))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    slots = torch.randperm(N + 4, generator=torch.Generator().manual_seed(1))[:N].to(torch.int32)
    slots[3], slots[7] = -1, N + 4  # outside the pool
    for alias in (False, True):
        s0 = x["s0"].clone()
        out = s0 if alias else torch.full_like(s0, 7.0)
        y = torch.full((T, D), 3.0, dtype=dtype, device="cuda")
        efla.efla_conv_fwd_varlen(x["x"], x["w"], cu, x["bias"], s0, slots.cuda(), y=y, s_final=out)
        want = x["s0"].clone() if alias else torch.full_like(s0, 7.0)
        at = 0
        for n, slot in zip(lens, slots.tolist()):
            inside = 0 <= slot < N + 4
            first = x["s0"][slot:slot + 1] if inside else None
            ry, rf = R.conv_ref(wide(x["x"][None, at:at + n]), wide(x["w"]), wide(x["bias"]), wide(first))
            if n:
                assert R.rel(y[None, at:at + n], ry) <= R.tol_conv(dtype), (n, slot)
            if inside:
                want[slot] = rf[0].to(dtype).cuda()
            at += n
        assert torch.equal(out, want)
        assert bool((y[at:] == 3.0).all())  # rows behind the last sequence
    made, none = efla.efla_conv_fwd_varlen(x["x"], x["w"], cu, x["bias"], want_final=False)
    assert none is None and bool((made[at:] == 0).all())


def test_packed_batch_of_many_sequences_and_malformed_offsets():
    N, D = 3000, 64
    lens = torch.randint(0, 4, (N,), generator=torch.Generator().manual_seed(0))
    T = int(lens.sum())
    x = dev(R.make_conv(N, 0, D, 4, BF, lead=(T,)))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).cuda()
    y, fin = efla.efla_conv_fwd_varlen(x["x"], x["w"], cu, x["bias"], x["s0"])
    state = x["s0"].double().cpu()
    full = x["x"].double().cpu()
    u = x["bias"].double().cpu().expand(T, D).clone()
    w, c = x["w"].double().cpu(), cu.tolist()
    for i in range(N):
        seq = torch.cat([state[i], full[c[i]:c[i + 1]]])
        for j in range(4):
            u[c[i]:c[i + 1]] += w[:, j] * seq[j:j + c[i + 1] - c[i]]
        state[i] = seq[len(seq) - 3:]
    assert R.rel(y, u / (1 + torch.exp(-u))) <= R.tol_conv(BF) and torch.equal(fin.double().cpu(), state)
    bad = torch.tensor([5, -3, 1 << 30, 2, 100, -7], dtype=torch.int32).cuda()  # numbers are unspecified, accesses are not
    efla.efla_conv_fwd_varlen(x["x"], x["w"], bad, x["bias"], x["s0"][:5].contiguous())
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W,D", [(2, 8), (3, 70), (4, 512), (4, 6144), (4, 1)])
def test_step_continues_the_forward(dtype, W, D):
    L, N = 9, 5
    x = dev(R.make_conv(N, L, D, W, dtype))
    y, fin = efla.efla_conv_fwd(x["x"], x["w"], x["bias"], x["s0"])
    st = x["s0"].clone()
    for t in range(L):
        out = efla.efla_conv_step(x["x"][:, t], x["w"], st, x["bias"])
        assert R.rel(out, y[:, t]) <= 2 * R.tol_conv(dtype)
    assert torch.equal(st, fin)
    pool = torch.randn(9, W - 1, D, device="cuda").to(dtype)
    keep, slots = pool.clone(), torch.tensor([4, -1, 0, 9, 8], dtype=torch.int32, device="cuda")
    given = torch.full((N, D), 5.0, dtype=dtype, device="cuda")
    out = efla.efla_conv_step(x["x"][:, 0], x["w"], pool, x["bias"], slots, y=given)
    made = efla.efla_conv_step(x["x"][:, 0], x["w"], keep.clone(), x["bias"], slots)
    for n, s in enumerate(slots.tolist()):
        if 0 <= s < 9:
            ry, rf = R.conv_ref(wide(x["x"][n:n + 1, :1]), wide(x["w"]), wide(x["bias"]), wide(keep[s:s + 1]))
            assert R.rel(out[n:n + 1, None], ry) <= R.tol_conv(dtype)
            assert torch.equal(pool[s].double().cpu(), rf[0]) and torch.equal(made[n], out[n])
        else:
            assert bool((out[n] == 5.0).all()) and bool((made[n] == 0).all())
    rest = [i for i in range(9) if i not in (4, 0, 8)]
    assert torch.equal(pool[rest], keep[rest])


def grads_ref(x, dy, dsf, act):
    ins = [None if x[n] is None else wide(x[n]).requires_grad_() for n in ("x", "w", "bias", "s0")]
    W = ins[1].shape[1]
    s0 = ins[0].new_zeros(x["x"].shape[0], W - 1, x["x"].shape[2]) if ins[3] is None else ins[3]
    y, fin = R.conv_ref(ins[0], ins[1], ins[2], s0, silu=act == "silu")
    loss = (y * wide(dy)).sum() + (0 if dsf is None else (fin * wide(dsf)).sum())
    want = [t for t in ins if t is not None]
    got = iter(torch.autograd.grad(loss, want, allow_unused=True))
    return [None if t is None else next(got) for t in ins]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,L,D", [(1, 1, 8), (2, 2, 24), (3, 5, 33), (2, 64, 512), (1, 259, 520), (2, 300, 37), (1, 1030, 64)])
def test_gradient(dtype, W, B, L, D):
    for full, act in ((True, "silu"), (False, None)):
        x = dev(R.make_conv(B, L, D, W, dtype, seed=L + W, s0=full, bias=full))
        gen = torch.Generator().manual_seed(9)
        dy = torch.randn(B, L, D, generator=gen).to(dtype).cuda()
        dsf = torch.randn(B, W - 1, D, generator=gen).to(dtype).cuda() if full else None
        dx, dw, db, ds0 = efla.efla_conv_bwd(x["x"], x["w"], dy, x["bias"], x["s0"], dsf, activation=act, want_ds0=full)
        rx, rw, rb, rs = grads_ref(x, dy, dsf, act)
        t = 2 * R.tol_conv(dtype)  # the terms' own errors, u's among them, and the result's rounding
        assert R.rel(dx, rx) <= t
        # terms' absolute sums: |x| |du| per tap, bounded through Cauchy-Schwarz by the norms over tokens
        scale_w = wide(x["x"]).flatten(0, 1).norm(dim=0) * wide(dy).flatten(0, 1).norm(dim=0) * 1.2
        scale_w = scale_w + (0 if x["s0"] is None else wide(x["s0"]).flatten(0, 1).norm(dim=0) * wide(dy).flatten(0, 1).norm(dim=0))
        sum_err = 32 * 2.0 ** -24 + (B * L) ** 0.5 * 2.0 ** -24
        assert R.rel(dw, rw, scale_w[:, None].expand(D, W)) <= sum_err
        if full:
            assert R.rel(db, rb, wide(dy).abs().sum((0, 1)) * 1.2) <= sum_err
            assert R.rel(ds0, rs) <= t
        else:
            assert db is None and ds0 is None


def test_gradient_in_wider_rows_and_of_no_tokens():
    x = dev(R.make_conv(2, 100, 64, 4, BF))
    dy = torch.randn(2, 100, 64, device="cuda").to(BF)
    want = efla.efla_conv_bwd(x["x"], x["w"], dy, x["bias"], x["s0"])
    for extra in (8, 5):
        rows = torch.full((2, 100, 64 + extra), 9.0, dtype=BF, device="cuda")
        got = efla.efla_conv_bwd(R.in_wider_rows(x["x"], 2, extra), x["w"], R.in_wider_rows(dy, 2, 8), x["bias"], x["s0"],
                                 dx=rows[..., :64])
        assert all(R.rel(a, b) <= R.tol_conv(BF) for a, b in zip(got, want)) and bool((rows[..., 64:] == 9.0).all())
        assert torch.equal(got[0], want[0])
    e = x["x"][:, :0]
    dsf = torch.randn(2, 3, 64, device="cuda").to(BF)
    dx, dw, db, ds0 = efla.efla_conv_bwd(e, x["w"], dy[:, :0], x["bias"], x["s0"], dsf)
    assert dx.shape == e.shape and not dw.any() and not db.any() and torch.equal(ds0, dsf)


def test_gradient_against_differences():
    x = R.make_conv(1, 6, 8, 4, F32)
    gen = torch.Generator().manual_seed(3)
    dy = torch.randn(1, 6, 8, generator=gen)
    got = efla.efla_conv_bwd(x["x"].cuda(), x["w"].cuda(), dy.cuda(), x["bias"].cuda(), x["s0"].cuda())
    for name, g in zip(("x", "w", "bias", "s0"), got):
        way = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        loss = []
        for sign in (1, -1):
            ins = {n: x[n].double() + (sign * 1e-5 * way if n == name else 0) for n in x}
            loss.append(float((R.conv_ref(ins["x"], ins["w"], ins["bias"], ins["s0"])[0] * dy).sum()))
        slope = (loss[0] - loss[1]) / 2e-5
        along = float((g.double().cpu() * way).sum())
        assert abs(slope - along) <= 1e-5 * float(g.double().norm().cpu() * way.norm())


def test_results_do_not_change_between_runs():
    x = dev(R.make_conv(2, 3000, 256, 4, BF))
    dy = torch.randn(2, 3000, 256, device="cuda").to(BF)
    first = efla.efla_conv_bwd(x["x"], x["w"], dy, x["bias"])
    for _ in range(3):
        again = efla.efla_conv_bwd(x["x"], x["w"], dy, x["bias"])
        assert all(torch.equal(a, b) for a, b in zip(first[:3], again[:3]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_another_stream_and_a_captured_graph(dtype):
    x = dev(R.make_conv(2, 300, 72, 4, dtype))
    dy = torch.randn(2, 300, 72, device="cuda").to(dtype)
    pool = torch.randn(4, 3, 72, device="cuda").to(dtype)
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5, 5, 290], dtype=torch.int32, device="cuda")

    def run():
        st = pool.clone()
        y, sf = efla.efla_conv_fwd(x["x"], x["w"], x["bias"], x["s0"])
        z = torch.zeros(300, 72, dtype=dtype, device="cuda")
        efla.efla_conv_fwd_varlen(x["x"][0], x["w"], cu, x["bias"], s0=st, slots=slots, y=z, s_final=st)
        t = torch.zeros(3, 72, dtype=dtype, device="cuda")
        efla.efla_conv_step(x["x"][0, :3], x["w"], st, x["bias"], slots=slots, y=t)
        return (y, sf, z, t, st) + tuple(efla.efla_conv_bwd(x["x"], x["w"], dy, x["bias"], s0=x["s0"]))

    def same(a, b):
        return all(p is r is None or torch.equal(p, r) for p, r in zip(a, b, strict=True))
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert same(want, got)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(run())
    for i in range(3):
        x["x"].copy_(torch.randn(2, 300, 72, device="cuda"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = run()
        assert all(same(want, got) for got in outs), i
