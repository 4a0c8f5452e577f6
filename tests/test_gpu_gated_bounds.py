"""Sizes at the ends of what the gated entry points and the plan accept, on the GPU."""
import ctypes

import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _gated as G

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


@pytest.mark.parametrize("chunk", [16, 32, 64])
@pytest.mark.parametrize("lens", [[TOP], [TOP - 15], [3, TOP - 63], [0, 5, TOP, 7], [2 ** 30] * 3], ids=str)
def test_plan_of_the_longest_requests(lens, chunk):
    """Offsets and order alone, by the C entry point: tables of their own size inside guarded arrays."""
    N, T, pad = len(lens), TOP, 128
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    cu = torch.full((pad + N + 1 + pad,), 77, dtype=torch.int32).cuda()
    order = torch.full((pad + N + pad,), 77, dtype=torch.int32).cuda()
    at = lambda t: ctypes.c_void_p(t.data_ptr() + 4 * pad)
    assert efla.lib().efla_pack_plan(ctypes.c_void_p(ln.data_ptr()), None, N, T, chunk, at(cu), at(order), None, None,
                                     ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    want = [0]
    for x in lens:
        want.append(min(want[-1] + x, T))
    n = [-(-(b - a) // chunk) for a, b in zip(want, want[1:])]
    assert cu[pad:-pad].tolist() == want
    assert order[pad:-pad].tolist() == sorted(range(N), key=lambda u: (-n[u], u))
    for t in (cu, order):
        assert bool((t[:pad] == 77).all()) and bool((t[-pad:] == 77).all())


def test_plan_of_the_largest_batch():
    """Through the binding, with the tables of 2^31 - 1 rows."""
    lens, starts = [9, TOP - 100], [4, 1000]
    p = efla.efla_pack_plan(torch.tensor(lens, dtype=torch.int32).cuda(), TOP, torch.tensor(starts, dtype=torch.int32).cuda())
    end = sum(lens)
    assert p.cu_seqlens.tolist() == [0, 9, end] and p.order.tolist() == [1, 0]
    rows = [0, 8, 9, 2 ** 30, end - 1, end, TOP - 1]
    assert p.token_seq[rows].tolist() == [0, 0, 1, 1, 1, -1, -1]
    wrap = lambda x: (x + 2 ** 31) % 2 ** 32 - 2 ** 31
    assert p.token_pos[rows].tolist() == [4, 12, 1000, wrap(2 ** 30 - 9 + 1000), wrap(end - 10 + 1000), -1, -1]


@pytest.mark.parametrize("N,H,chunk", [(4096, 32, 64), (2048, 16, 16)])
def test_packed_batch_of_many_long_requests(N, H, chunk):
    """2^20 tokens in thousands of sequences: each gives, bit for bit, what it gives alone."""
    T, d, n = 2 ** 20, 128, 2 ** 20 // N
    gen = torch.Generator(device="cuda").manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    k = r(T, 1, d)
    x = [r(T, 1, d).to(torch.bfloat16), (k / k.norm(dim=-1, keepdim=True)).to(torch.bfloat16),
         torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen),
         torch.sigmoid(r(T, H)).to(torch.bfloat16), -0.02 * r(T, H).exp()]
    cu = torch.arange(0, T + 1, n, dtype=torch.int32).cuda()
    o, S = efla.efla_gated_chunk_fwd_varlen(*x, cu, chunk=chunk)
    for u in (0, 1, N // 2, N - 1):
        o1, S1 = efla.efla_gated_chunk_fwd(*(t[None, u * n:(u + 1) * n].contiguous() for t in x), chunk=chunk)
        assert torch.equal(o[u * n:(u + 1) * n], o1[0]) and torch.equal(S[u], S1[0])


def test_largest_batches_that_run():
    """65536 requests of 16 heads (64 GiB of states): one token each through the packed forward, 3.8e9 threads in one
    launch, then a decode step; some of them against themselves alone."""
    N, H, d = 65536, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    k = r(2, N, 1, d)
    x = [r(2, N, 1, d).bfloat16(), (k / k.norm(dim=-1, keepdim=True)).bfloat16(), r(2, N, H, d).bfloat16(),
         torch.sigmoid(r(2, N, H)).bfloat16(), -0.02 * r(2, N, H).exp()]
    cu = torch.arange(N + 1, dtype=torch.int32).cuda()
    o, S = efla.efla_gated_chunk_fwd_varlen(*(t[0] for t in x), cu)
    rows = [0, 1, 9, 4097, 40000, N - 2, N - 1]
    few = [t[:, rows].contiguous() for t in x]
    # at d_k 128 a batch this small takes the float32 recurrence: the two agree to the chunked passes' tolerance
    o1, S1 = efla.efla_gated_chunk_fwd_varlen(*(t[0] for t in few), torch.arange(len(rows) + 1, dtype=torch.int32).cuda())
    assert G.rel(o[rows], o1) <= 2 * G.tol_o(torch.bfloat16, 1, d) and G.rel(S[rows], S1) <= 2 * G.tol_s(torch.bfloat16, 1, d)
    S1 = S[rows].clone()
    y = efla.efla_gated_step(*(t[1] for t in x), S)
    y1 = efla.efla_gated_step(*(t[1] for t in few), S1)
    # The few rows take value blocks of 32 columns, the many of 64: a column's d_k products are then summed in 32 parts
    # of 4 and in 16 of 8, so the sums round differently; each is within tol32 of the exact one, y one rounding more.
    assert G.rel(y[rows], y1) <= 2 * (2.0 ** -8 + G.tol32(1, d)) and G.rel(S[rows], S1) <= 2 * G.tol32(1, d)
