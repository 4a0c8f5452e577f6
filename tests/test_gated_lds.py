"""LDS arrays that are read or written 16 bytes at a time are declared with that
alignment, rather than left to what the compiler aligns arrays to (source check)."""
import glob
import os
import re

import pytest

from delta_rule_sequence_efla_amd import build

VECTORS = r"(?:f32x4|i32x4|u32x4|bf16x8)"


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(build.CSRC, "gated*")) + [os.path.join(build.CSRC, "plan.hip")]),
                         ids=os.path.basename)
def test_arrays_used_in_16_byte_pieces_declare_it(path):
    with open(path) as f:
        src = f.read()
    # one array name per declarator, with the declaration's first line
    arrays = {}
    for decl in re.findall(r"__shared__[^;]*;", src):
        for name in re.findall(r"(\w+)\[", decl):
            arrays.setdefault(name, []).append(decl)
    used = set(re.findall(r"reinterpret_cast<(?:const )?" + VECTORS + r"\*>\(&?(\w+)", src)) & set(arrays)
    bad = [n for n in used if not all("__align__(16)" in d or "__align__(1024)" in d for d in arrays[n])]
    assert not bad, bad
    if path.endswith("gated_step.hip"):
        assert {"us", "red_k", "red_q", "cS", "dS"} <= used
