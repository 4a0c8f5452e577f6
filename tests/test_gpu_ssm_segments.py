"""Scans of few, long sequences, which the forward pass cuts into segments: against the
64-bit form, and over the states that they started from."""
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


def cut(B, H, Hk, L, dk, dv, dtype):
    return efla.efla_ssm_fwd_workspace_size(B, H, Hk, L, dk, dv, dtype) > 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,H,Hk,dk,dv", [(1, 1100, 2, 1, 64, 64), (1, 1025, 2, 2, 128, 32), (2, 3000, 1, 1, 64, 128),
                                            (3, 1601, 2, 1, 128, 64)])
def test_dense(dtype, B, L, H, Hk, dk, dv):
    assert cut(B, H, Hk, L, dk, dv, dtype)
    for s0 in (True, False):
        x = dev(R.make_scan(B, L, H, Hk, dk, dv, dtype, seed=L, s0=s0, steps=(1e-4, 0.1)))
        a, kw = ins(x)
        o, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        ro, rs = R.scan_ref(*(None if t is None else t.cpu() for t in R.wide(x)))
        assert R.rel(o, ro) <= R.tol_o(dtype, L, dk) and R.rel(S, rs) <= R.tol_s(dtype, L, dk)
        if s0:
            st = x["s0"].clone()
            o2, S2 = efla.efla_ssm_fwd(*a, s0=st, s_final=st, **kw)
            assert S2 is st and torch.equal(o, o2) and torch.equal(S, st)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1500, 0, 7], [0, 0, 2000], [64, 1200, 65], [700, 700, 700, 1], [3000], [1, 1, 1, 1800]])
def test_packed(dtype, lens):
    N, T, H, Hk, dk, dv = len(lens), sum(lens) + 5, 2, 1, 64, 64
    assert efla.efla_ssm_fwd_varlen_workspace_size(N, H, Hk, T, dk, dv, dtype) > 0
    x = dev(R.make_scan(N + 2, 0, H, Hk, dk, dv, dtype, lead=(T,), steps=(1e-4, 0.1)))
    a, kw = ins(x)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    slots = torch.arange(N, 0, -1, dtype=torch.int32)
    pool = x["s0"].clone()
    o = torch.full((T, H, dv), 3.0, dtype=dtype, device="cuda")
    efla.efla_ssm_fwd_varlen(*a, cu, s0=pool, slots=slots.cuda(), o=o, s_final=pool, **kw)
    at = 0
    for n, slot in zip(lens, slots.tolist()):
        part = {m: x[m][None, at:at + n] for m in ("q", "k", "v", "dt")}
        part.update({m: x[m] for m in ("a", "d", "bias")}, s0=x["s0"][slot:slot + 1])
        ro, rs = R.scan_ref(*(None if t is None else t.cpu() for t in R.wide(part)))
        if n:
            assert R.rel(o[None, at:at + n], ro) <= R.tol_o(dtype, n, dk)
        assert R.rel(pool[slot:slot + 1], rs) <= R.tol_s(dtype, n, dk)
        at += n
    assert bool((o[at:] == 3.0).all()) and torch.equal(pool[0], x["s0"][0]) and torch.equal(pool[N + 1], x["s0"][N + 1])
    none = torch.full_like(slots, -1)  # no state named: from zero, none written
    keep = pool.clone()
    efla.efla_ssm_fwd_varlen(*a, cu, s0=pool, slots=none.cuda(), o=o, s_final=pool, **kw)
    assert torch.equal(pool, keep)
    bad = torch.tensor([5, -3, 1 << 30, 2, 100, -7], dtype=torch.int32).cuda()[:N + 1].contiguous()
    efla.efla_ssm_fwd_varlen(*a, bad, **kw)  # numbers are unspecified, accesses are not
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_graph_and_two_calls_at_once(dtype):
    x = dev(R.make_scan(1, 1500, 2, 1, 64, 64, dtype))
    a, kw = ins(x)
    want, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(efla.efla_ssm_fwd(*a, s0=x["s0"], **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(t, S) for o, t in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, t = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    for _ in range(3):
        x["v"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        want, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
        assert torch.equal(o, want) and torch.equal(t, S)


def test_a_nan_behind_a_segment():
    x = dev(R.make_scan(2, 2000, 1, 1, 64, 64, BF))
    a, kw = ins(x)
    want, S = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    x["v"][0, 1000] = float("nan")
    o, t = efla.efla_ssm_fwd(*a, s0=x["s0"], **kw)
    assert torch.equal(o[1], want[1]) and torch.equal(t[1], S[1])
    assert torch.equal(o[0, :960], want[0, :960]) and bool(o[0, 1000].isnan().any())
