"""Rows that no request and no sequence writes, in outputs that the binding makes,
with the allocator's memory full of NaN beforehand; and in captured graphs."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _gated as G
from tests.test_gpu_gated import _graph, dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def poison(like):
    torch.full_like(like, float("nan"))  # freed at once: the next tensor of its size takes its place


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_step_skipped_rows(dt):
    x = dev(G.make(5, 1, 4, 2, 64, 64, dt, seed=1, s0=False))
    a = [x[n][:, 0].contiguous() for n in G.NAMES]
    pool = torch.randn(4, 4, 64, 64, generator=torch.Generator().manual_seed(2)).cuda()
    slots = torch.tensor([3, -1, 0, 4, 2], dtype=torch.int32).cuda()
    want = efla.efla_gated_step(*(t[[0, 2, 4]].contiguous() for t in a), pool[[3, 0, 2]].contiguous())
    poison(a[2])
    o = efla.efla_gated_step(*a, pool.clone(), slots=slots)
    assert torch.equal(o[[0, 2, 4]], want) and not bool(o[[1, 3]].any())

    def run():
        return efla.efla_gated_step(*a, pool.clone(), slots=slots)

    gr, out = _graph(run)
    for live in ([3, -1, 0, 4, 2], [-1, 1, -1, 9, 0], [0, 1, 2, 3, -7]):
        slots.copy_(torch.tensor(live, dtype=torch.int32))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run())
        rest = [i for i, s in enumerate(live) if not 0 <= s < 4]
        assert not bool(out[rest].any()) and bool(out[[i for i in range(5) if i not in rest]].any())


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_packed_rows_of_no_sequence(dt):
    T = 300
    x = dev(G.make(2, 0, 4, 2, 64, 64, dt, seed=3, lead=(T,)))
    a = [x[n] for n in G.NAMES]
    cu = torch.tensor([7, 60, 250], dtype=torch.int32).cuda()
    poison(a[2])
    o, S = efla.efla_gated_chunk_fwd_varlen(*a, cu, x["s0"])
    assert not bool(o[:7].any()) and not bool(o[250:].any()) and bool(o.isfinite().all())
    given = torch.full_like(o, 7.0)
    efla.efla_gated_chunk_fwd_varlen(*a, cu, x["s0"], o=given)
    assert torch.equal(given[7:250], o[7:250]) and bool((given[:7] == 7).all())
