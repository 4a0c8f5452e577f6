"""dg in a type of its own: what the C ABI and the binding refuse (CPU)."""
import ctypes

import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests.test_gated_checks import host, inputs  # noqa: F401  (host: the fixture)

BF, F32 = torch.bfloat16, torch.float32
OK, INVALID, WORKSPACE = 0, 1, 3
F = ctypes.c_void_p(4096)


def bwd(dtype, dg, L=640, ws=None):
    return efla.lib().efla_gated_chunk_bwd_typed(F, F, F, F, F, None, F, None, F, F, F, F, F, None, 1, 4, 2, L, 64, 64, 64, dtype,
                                                 dg, 0, ws, 0, None)


def test_types_of_dg():
    f32, bf = 0, 1
    assert bwd(bf, bf) == bwd(bf, f32) == bwd(f32, f32) == WORKSPACE  # accepted up to the missing workspace
    assert bwd(f32, bf) == bwd(bf, 7) == bwd(f32, -1) == INVALID
    assert bwd(bf, f32, L=0) == OK


def test_binding_refuses(host):  # noqa: F811
    for dt, bad in ((BF, torch.float16), (BF, torch.float64), (F32, BF), (F32, torch.int32)):
        a = inputs((2, 8), dt=dt)
        with pytest.raises(ValueError):
            efla.efla_gated_chunk_bwd(*a, torch.zeros_like(a[2]), dg_dtype=bad)
