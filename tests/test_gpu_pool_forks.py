"""Rows copied to many others: every byte, on both sides of the rule that lets copies share
a read, and the time of wide forks beside that of as many copies of distinct rows."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def sources(kind, N, parents, gen):
    i = torch.arange(N)
    return {"grouped": i * parents // N, "in turn": i % parents, "random": torch.randint(0, parents, (N,), generator=gen)}[kind]


@pytest.mark.parametrize("kind", ["grouped", "in turn", "random"])
@pytest.mark.parametrize("N,parents", [(1, 1), (9, 1), (10, 2), (64, 1), (65, 1), (66, 3), (130, 1), (200, 20), (500, 1),
                                       (500, 7), (512, 60), (513, 2)])
def test_every_copy(kind, N, parents):
    gen = torch.Generator().manual_seed(N + parents)
    P = N + parents + 3
    # rows of 32 MiB / N and a little, so that lists of up to 512 share their reads, and small ones, which do not
    for width in (((32 << 20) // N // 4 + 63) // 64 * 64 + 4, 12):
        pool = torch.randn(P, width, device="cuda")
        src, dst = sources(kind, N, parents, gen) + N, torch.randperm(N, generator=gen)
        src[torch.rand(N, generator=gen) < 0.05] = -1     # cleared
        dst[torch.rand(N, generator=gen) < 0.2] = P + 5   # nothing
        src, dst = src.to(**I32), dst.to(**I32)
        want, live = pool.clone(), dst < P
        rows = torch.where((src >= 0)[:, None], pool[src.clamp(min=0)], 0)
        want[dst[live].long()] = rows[live]
        del rows
        efla.efla_pool_copy([pool], src, dst)
        assert torch.equal(pool, want), (width, (pool != want).any(1).nonzero().flatten().tolist()[:10])


@pytest.mark.parametrize("kib,N,times", [(4, 500, 2.0), (64, 500, 2.0), (256, 500, 1.5), (64, 256, 2.0)])
def test_the_time_of_wide_forks(kib, N, times):
    """One row to N others reads less than N distinct rows to N others, and may not take `times` as long."""
    pool = torch.randn(2 * N, kib * 256, device="cuda")
    dst = torch.randperm(N, generator=torch.Generator().manual_seed(0)).to(**I32)
    one, each = torch.full((N,), N, **I32), torch.arange(N, 2 * N, **I32)
    took = {0: [], 1: []}
    for _ in range(9):
        for which, src in enumerate((one, each)):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(20):
                efla.efla_pool_copy([pool], src, dst)
            end.record()
            torch.cuda.synchronize()
            took[which].append(start.elapsed_time(end) * 50)
    fork, copies = (sorted(took[i])[4] for i in (0, 1))
    assert fork <= times * copies, (fork, copies)
