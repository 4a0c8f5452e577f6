"""The convolution over many tokens, forward, packed and gradient, against a form in 64 bits
over all tokens at once.  The gradient takes runs of 8 to 64 tokens a wavefront, the longest that leave 2048
wavefronts; the forward pass 8, and more where the launch would have 2^32 threads."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def run_of(B, L, D):
    return next((r for r in (64, 32, 16) if B * -(-L // r) * -(-D // 512) >= 2048), 8)


def make(lead, D, W, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    return n(*lead, D).to(dtype), (0.5 * n(D, W)).to(dtype), (0.5 * n(D)).to(dtype), n


FORWARD = [(1, 262161, 40), (3, 87399, 24), (2, 262201, 40), (1, 1048641, 8), (5, 209800, 16), (2, 8199, 4101)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,D", FORWARD)
def test_forward(dtype, B, L, D):
    x, w, bias, n = make((B, L), D, 4, dtype, L)
    s0 = n(B, 3, D).to(dtype)
    y, fin = efla.efla_conv_fwd(x, w, bias, s0)
    for b in range(B):
        ry, rf = R.conv_ref(x[b:b + 1].double(), w.double(), bias.double(), s0[b:b + 1].double())
        assert R.rel(y[b:b + 1], ry) <= R.tol_conv(dtype)
        # no single value wrong among the many: a sum of five terms of up to about 3, off by 32 half steps of it
        worst = ((y[b:b + 1].double() - ry).abs() / (1 + ry.abs())).max()
        assert float(worst) <= 16 * R.tol_conv(dtype) and torch.equal(fin[b:b + 1].double(), rf)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,D,W,longest", [(262300, 40, 4, 9), (262300, 40, 3, 200), (524500, 24, 4, 100), (1048800, 8, 4, 40),
                                           (1048800, 8, 2, 70000)])
def test_packed(dtype, T, D, W, longest):
    """Short and empty sequences inside one run, and rows of none behind the last."""
    gen = torch.Generator().manual_seed(T + W)
    lens = torch.randint(0, longest + 1, (2 * T // longest + 8,), generator=gen)
    lens[torch.rand(len(lens), generator=gen) < 0.1] = 0
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    cu = cu[cu <= T - 5]
    N, used = len(cu) - 1, int(cu[-1])
    x, w, bias, n = make((T,), D, W, dtype, T)
    pool, slots = n(N + 2, W - 1, D).to(dtype), torch.randperm(N + 2, generator=gen)[:N]
    y, out = torch.full_like(x, 3.0), torch.full_like(pool, 7.0)
    efla.efla_conv_fwd_varlen(x, w, cu.to(torch.int32).cuda(), bias, pool, slots.to(torch.int32).cuda(), y=y, s_final=out)
    cu, slots = cu.cuda(), slots.cuda()
    # every sequence's state and tokens in one tensor: token t of sequence i at t + (W - 1) (i + 1)
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), cu[1:] - cu[:-1])
    at = torch.arange(used, device="cuda") + (W - 1) * (seq + 1)
    full = torch.zeros(used + (W - 1) * N, D, dtype=torch.float64, device="cuda")
    full[at] = x[:used].double()
    first = (cu[:-1] + (W - 1) * torch.arange(N, device="cuda"))[:, None] + torch.arange(W - 1, device="cuda")
    full[first] = pool[slots].double()
    u = bias.double() + sum(w.double()[:, j] * full[at - (W - 1) + j] for j in range(W))
    ry = u / (1 + torch.exp(-u))
    assert R.rel(y[:used], ry) <= R.tol_conv(dtype) and bool((y[used:] == 3.0).all())
    assert float(((y[:used].double() - ry).abs() / (1 + ry.abs())).max()) <= 16 * R.tol_conv(dtype)
    last = (cu[1:] + (W - 1) * torch.arange(N, device="cuda"))[:, None] + torch.arange(W - 1, device="cuda")
    assert torch.equal(out[slots].double(), full[last])
    rest = torch.ones(N + 2, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert bool((out[rest] == 7.0).all())


@pytest.mark.parametrize("L,packed", [(2 ** 29 + 77, False), (2 ** 30 + 5, True), (2 ** 31 - 9, False)])
def test_launches_of_2_32_threads(L, packed):
    """One channel, whose rows a wavefront moves one by one: runs of 16, 32 and 64 tokens."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(L, 1, dtype=BF, device="cuda")
    step = 1 << 27
    for at in range(0, L, step):
        x[at:at + step] = torch.randn(min(step, L - at), 1, generator=gen, device="cuda").to(BF)
    w, bias = torch.tensor([[0.3, -0.5, 0.25, 0.75]], device="cuda").to(BF), torch.tensor([0.125], device="cuda").to(BF)
    state = torch.randn(3, 3, 1, generator=gen, device="cuda").to(BF)
    cuts = [0, 5 * step + 3, L - 4] if packed else [0, L]  # two sequences and rows of none
    if packed:
        y, fin = torch.full_like(x, 3.0), None
        _, fin = efla.efla_conv_fwd_varlen(x, w, torch.tensor(cuts, dtype=torch.int32, device="cuda"), bias, state[:2].contiguous(), y=y)
        assert bool((y[cuts[-1]:] == 3.0).all())
    else:
        y, fin = efla.efla_conv_fwd(x[None], w, bias, state[:1].contiguous())
        y = y[0]
    wd = w[0].double()
    for i, (first, end) in enumerate(zip(cuts, cuts[1:])):
        assert torch.equal(fin[i], x[end - 3:end])
        for at in range(first, end, step):
            n = min(step, end - at)
            full = torch.cat([state[i] if at == first else x[at - 3:at], x[at:at + n]])[:, 0].double()
            u = bias.double() + sum(wd[j] * full[j:j + n] for j in range(4))
            ry = u / (1 + torch.exp(-u))
            assert R.rel(y[at:at + n, 0], ry) <= R.tol_conv(BF), (i, at)
            del full, u, ry


GRADIENT = [(2, 17001, 72, 16), (1, 32771, 512, 16), (3, 11003, 37, 16), (2, 33333, 72, 32), (1, 65601, 40, 32),
            (2, 66001, 24, 64), (8, 2049, 4096, 64), (1, 131073, 33, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,D,run", GRADIENT)
def test_gradient(dtype, B, L, D, run):
    """dx and ds0 as in the short gradients.  dw and dbias are sums of B L terms: each is off by half a step of the
    absolute sum for its factors' 32 roundings, and by sqrt(B L) of the terms' root of squares for the summation."""
    assert run_of(B, L, D) == run
    W = 4
    x, w, bias, n = make((B, L), D, W, dtype, L)
    s0, dy, dsf = n(B, 3, D).to(dtype), n(B, L, D).to(dtype), n(B, 3, D).to(dtype)
    dx, dw, db, ds0 = efla.efla_conv_bwd(x, w, dy, bias, s0, dsf)
    rw, rb = torch.zeros(D, W, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    scale_w, scale_b = torch.zeros_like(rw), torch.zeros_like(rb)
    wd = w.double()
    for b in range(B):
        full = torch.cat([s0[b], x[b]]).double()
        u = bias.double() + sum(wd[:, j] * full[j:j + L] for j in range(W))
        sg = 1 / (1 + torch.exp(-u))
        du = dy[b].double() * (sg + u * sg * (1 - sg))
        rx = torch.cat([torch.zeros(L, D, dtype=torch.float64, device="cuda"), dsf[b].double()])
        for j in range(W):
            rx[j:j + L] += wd[:, j] * du
            rw[:, j] += (full[j:j + L] * du).sum(0)
            scale_w[:, j] += (full[j:j + L] * du).abs().sum(0)
        rb += du.sum(0)
        scale_b += du.abs().sum(0)
        t = 2 * R.tol_conv(dtype)
        assert R.rel(dx[b], rx[3:]) <= t and R.rel(ds0[b], rx[:3]) <= t
        assert float(((dx[b].double() - rx[3:]).abs() / (1 + rx[3:].abs())).max()) <= 16 * t
    # a term may be off by its u, too: 16 half steps of |x dy|, of which |x du| is a part
    bound = 64 * 2.0 ** -24 + (B * L) ** 0.5 * 2.0 ** -24
    assert bool(((dw.double() - rw).abs() <= bound * scale_w).all()) and bool(((db.double() - rb).abs() <= bound * scale_b).all())
    again = efla.efla_conv_bwd(x, w, dy, bias, s0, dsf)
    assert all(torch.equal(p, r) for p, r in zip((dx, dw, db, ds0), again))
