"""Sizes at the ends of what the gated entry points and the plan accept, on the CPU."""
import ctypes
import os
import subprocess

import pytest
import torch

from delta_rule_sequence_efla_amd import build, efla

COUNTS = r"""
#include "gated.h"
#include <stdio.h>
#include <stdlib.h>
int main(int n, char** a) {
  for (int i = 2; i < n; ++i) printf("%d\n", efla::chunk_count(atoi(a[i]), atoi(a[1])));
}
"""


@pytest.mark.parametrize("shift", [4, 5, 6])
def test_chunk_counts_up_to_the_last_length(tmp_path, shift):
    """The plan orders requests by this count (host build of the same function): one request of
    2^31 - 1 tokens must not count as fewer than the -1 its table is padded with."""
    src = tmp_path / "counts.hip"
    src.write_text(COUNTS)
    exe = str(tmp_path / "counts")
    subprocess.run([build.HIPCC, f"--offload-arch={build.ARCH}", "--cuda-host-only", "-std=c++17", f"-I{build.CSRC}",
                    str(src), "-o", exe], check=True, capture_output=True)
    chunk, top = 1 << shift, 2 ** 31 - 1
    n = [0, 1, chunk - 1, chunk, chunk + 1, top - chunk, top - chunk + 1, top - chunk + 2, top - 1, top]
    got = subprocess.run([exe, str(shift), *map(str, n)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == [-(-x // chunk) for x in n]
    # and it is what the plan's kernel counts with
    with open(os.path.join(build.CSRC, "plan.hip")) as f:
        assert "chunk_count(end[u]" in f.read()


# ---------------------------------------------------- packed batches of many sequences and tokens
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
NUL, FAKE = None, ctypes.c_void_p(4096)


def varlen(N, H, T, chunk=64, Hk=1, d=128, dt=1):
    """Status of a packed call whose workspace is missing: WORKSPACE once the shape is accepted."""
    return efla.lib().efla_gated_chunk_fwd_varlen(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, NUL, NUL, N, N, NUL, FAKE, NUL, H, Hk, T,
                                                  d, d, chunk, dt, 0, NUL, 0, NUL)


def test_packed_batches_are_bounded_by_what_runs():
    """2048 and 4096 sequences in 2^20 tokens: T / 64 + N chunk slots a head whatever chunk is named, 12 KiB of X
    and 1 KiB of gates each, and 4 bytes a sequence for the schedule."""
    size = efla.efla_gated_chunk_fwd_varlen_workspace_size
    for N, H in ((2048, 16), (4095, 32), (4096, 32), (4097, 32), (65536, 16)):
        want = H * (2 ** 20 // 64 + N) * 13 * 1024 + (4 * N + 255) // 256 * 256
        for chunk in (16, 32, 64):
            assert size(N, H, 1, 2 ** 20, 128, 128, chunk, torch.bfloat16) == want
            assert varlen(N, H, 2 ** 20, chunk) == WORKSPACE
    # the largest T, in one sequence and in many
    assert size(1, 1, 1, 2 ** 31 - 1, 64, 64, 16, torch.bfloat16) == (2 ** 25 - 1 + 1) * 13 * 1024 + 256
    assert varlen(1, 1, 2 ** 31 - 1, 16, d=64) == WORKSPACE


def test_packed_batches_beyond_the_grid_are_refused():
    size = efla.efla_gated_chunk_fwd_varlen_workspace_size
    for N, H, T in ((2 ** 28, 1, 640), (2 ** 20, 2 ** 8, 640), (1, 2 ** 7, 2 ** 31 - 1)):  # workgroups, workgroups, slots
        assert size(N, H, 1, T, 128, 128, 64, torch.bfloat16) == 0 and varlen(N, H, T) == UNSUPPORTED
    for bad in (dict(N=-1), dict(T=-1), dict(T=2 ** 31), dict(H=0), dict(Hk=0), dict(H=4, Hk=3), dict(dt=5)):
        assert varlen(**{**dict(N=2, H=4, T=640), **bad}) == INVALID
    assert size(0, 4, 2, 640, 64, 64, 64, torch.bfloat16) == 0


# ----------------------------------------------------------- launches of 2^32 threads and more
def dense(B, H, L, dt=1, d=128, bwd=False):
    """Status of a dense call without pointers: INVALID once the sizes are accepted."""
    n = [NUL] * (14 if bwd else 8)
    if bwd:
        n[-1] = FAKE  # ds0
    f = efla.lib().efla_gated_chunk_bwd if bwd else efla.lib().efla_gated_chunk_fwd
    return f(*n, B, H, 1, L, d, d, 64, dt, 0, NUL, 0, NUL)


def step(N, H, d=128):
    return efla.lib().efla_gated_step(NUL, NUL, NUL, NUL, NUL, NUL, NUL, NUL, N, N, H, 1, d, d, 1, 0, NUL)


def test_launches_of_2_to_32_threads_are_refused():
    """A workgroup has 896 threads per 32 value columns in the chunked forward at d_k 128, 512 or 832 per 16 in the
    recurrence, 576 per 32 for each of the backward's two chains, 256 per 64 in the step."""
    bf, f32 = 1, 0
    top = (2 ** 32 - 1) // (4 * 896)
    assert dense(top, 1, 500) == INVALID and dense(top + 1, 1, 500) == UNSUPPORTED
    assert varlen(top, 1, 2 ** 24) == WORKSPACE and varlen(top + 1, 1, 2 ** 24) == UNSUPPORTED
    for L, threads in ((1, 512), (300, 832)):
        top = (2 ** 32 - 1) // (8 * threads)
        assert dense(top, 1, L, f32) == INVALID and dense(top + 1, 1, L, f32) == UNSUPPORTED
    top = (2 ** 32 - 1) // (2 * 4 * 576)
    assert dense(top, 1, 20, bwd=True) == INVALID and dense(top + 1, 1, 20, bwd=True) == UNSUPPORTED
    assert step(2 ** 20 - 1, 8) == INVALID and step(2 ** 20, 8) == UNSUPPORTED
    size, sizeb = efla.efla_gated_chunk_fwd_workspace_size, efla.efla_gated_chunk_bwd_workspace_size
    assert size(65536, 32, 1, 500, 128, 128, 64, torch.bfloat16) == sizeb(65536, 32, 1, 500, 128, 128, 64, torch.bfloat16) == 0
    assert size(65536, 16, 1, 500, 128, 128, 64, torch.bfloat16) > 0
