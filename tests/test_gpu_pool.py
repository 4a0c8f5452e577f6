"""Moves of state-pool rows on the GPU: every byte as the plain form leaves it."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def make(P, shapes, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(P, *s, generator=gen, device="cuda").to(t) for s, t in shapes]


SHAPES = [((4, 16, 16), torch.float32), ((3, 100), torch.bfloat16), ((3, 7), torch.bfloat16), ((5,), torch.float32),
          ((2, 128, 128), torch.float32), ((1,), torch.bfloat16)]


@pytest.mark.parametrize("P,src,dst", [
    (6, [0, 0, 3, -1, 9], [1, 2, 4, 5, 3]),
    (9, [5], [0]),
    (9, [-1, -1, 100], [0, 8, 4]),
    (40, [1] * 19 + [2] * 15, list(range(5, 39))),
    (6, [0, 1, 2], [-1, 6, 5]),
])
def test_copy(P, src, dst):
    pools = make(P, SHAPES)
    want = [p.clone() for p in pools]
    for s, d in zip(src, dst):
        if 0 <= d < P:
            for w, p in zip(want, pools):
                w[d] = p[s] if 0 <= s < P else 0
    efla.efla_pool_copy(pools, torch.tensor(src, **I32), torch.tensor(dst, **I32))
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


def test_many_pools_and_rows():
    P = 300
    pools = make(P, [((65,), torch.bfloat16)] * 70 + [((32,), torch.float32)] * 70)  # three launches
    want = [p.clone() for p in pools]
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(0))
    src, dst = perm[:150][torch.randint(0, 40, (150,))], perm[150:]
    for w in want:
        w[dst.cuda()] = w[src.cuda()]
    efla.efla_pool_copy(pools, src.to(**I32), dst.to(**I32))
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


def compact(P, slots, shapes=SHAPES, in_place=False):
    pools = make(P, shapes)
    want = [p.clone() for p in pools]
    new, moves, K = R.compact_ref(slots, P)
    for s, d in moves:
        for w, p in zip(want, pools):
            w[d] = p[s]
    t = torch.tensor(slots, **I32)
    got, live = efla.efla_pool_compact(pools, t, new_slots=t if in_place else None)
    assert got.tolist() == new and live.tolist() == [K]
    assert in_place or t.tolist() == slots
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


@pytest.mark.parametrize("P,slots", [
    (5, [4, 2]), (5, [0, 1, 2]), (5, [4, 3, 2, 1, 0]), (5, [-1, 9]), (5, [4]), (1, [0]), (7, [6, 6, -1, 6, 2]),
    (64, [63, 32, 31, 0, -1, 64]), (33, [32]), (12, [11, 10, 9, 8, 7, 6])])
def test_compact(P, slots):
    compact(P, slots)
    compact(P, slots, in_place=True)


def test_compact_of_many_rows():
    gen = torch.Generator().manual_seed(3)
    for P, n in ((131072, 5000), (5000, 4999), (1025, 600), (1024, 1), (70000, 69000)):
        slots = torch.randperm(P, generator=gen)[:n].tolist()
        compact(P, slots, [((3,), torch.float32)])


def test_no_entries_and_a_captured_graph():
    pools = make(8, SHAPES)
    keep = [p.clone() for p in pools]
    none = torch.empty(0, **I32)
    efla.efla_pool_copy(pools, none, none)
    new, live = efla.efla_pool_compact(pools, none)
    assert new.numel() == 0 and live.tolist() == [0] and all(torch.equal(p, k) for p, k in zip(pools, keep))
    slots = torch.tensor([7, 5, 1, -1], **I32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new, live = efla.efla_pool_compact(pools, slots)
        efla.efla_pool_copy(pools, new[2:3], slots[:1])
    for order in ([7, 5, 1, -1], [3, -1, 6, 0], [0, 1, 2, 3]):
        for p, k in zip(pools, keep):
            p.copy_(k)
        slots.copy_(torch.tensor(order, **I32))
        graph.replay()
        torch.cuda.synchronize()
        want_new, moves, K = R.compact_ref(order, 8)
        assert new.tolist() == want_new and live.tolist() == [K]
        for p, k in zip(pools, keep):
            w = k.clone()
            for s, d in moves:
                w[d] = k[s]
            row = w[want_new[2]].clone()
            w[order[0]] = row
            assert torch.equal(p, w)


@pytest.mark.parametrize("N", [512, 513, 3000])
def test_forks_of_long_lists(N):
    """Lists on both sides of the length up to which one read serves all copies of a row."""
    P = N + 40
    pool = torch.randn(P, 24, device="cuda")
    gen = torch.Generator().manual_seed(N)
    src = torch.randint(-1, 40, (N,), generator=gen)
    src[src >= 0] += N  # the last 40 rows, or none: cleared
    dst = torch.randperm(N, generator=gen)
    want = pool.clone()
    want[dst.cuda()] = torch.where((src >= 0).cuda()[:, None], pool[src.clamp(min=0).cuda()], torch.zeros((), device="cuda"))
    efla.efla_pool_copy([pool], src.to(**I32), dst.to(**I32))
    assert torch.equal(pool, want)
