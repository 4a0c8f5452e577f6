"""Sizes at the ends of what the gated entry points and the plan accept, on the CPU."""
import os
import subprocess

import pytest

from delta_rule_sequence_efla_amd import build

COUNTS = r"""
#include "common.h"
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
