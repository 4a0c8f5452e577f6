"""Outputs that the gated binding makes itself hold nothing of the allocator's: rows
that no request and no sequence writes are zero (CPU, with the library replaced by
one that writes nothing)."""
import pytest
import torch

from delta_rule_sequence_efla_amd import efla

BF = torch.bfloat16


class _Writes:
    """A library whose calls succeed and write nothing."""

    def __getattr__(self, name):
        return (lambda *a: 0)


@pytest.fixture
def host(monkeypatch):
    monkeypatch.setattr(efla, "_same", lambda *a: None)
    monkeypatch.setattr(efla, "lib", lambda: _Writes())
    monkeypatch.setattr(efla, "_call", lambda fn, index, where, *a: fn(*a))
    made = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: made(t, **k).fill_(float("nan")))
    efla._gated_workspace.cache_clear()
    yield
    efla._gated_workspace.cache_clear()


def inputs(n, H=4, Hk=2, dk=16, dv=32):
    q = torch.zeros(n, Hk, dk, dtype=BF)
    return [q, q.clone(), torch.zeros(n, H, dv, dtype=BF), torch.zeros(n, H, dtype=BF), torch.zeros(n, H)]


def test_step_with_slots(host):
    o = efla.efla_gated_step(*inputs(3), torch.zeros(7, 4, 16, 32), slots=torch.tensor([2, -1, 9], dtype=torch.int32))
    assert o.dtype == BF and o.shape == (3, 4, 32) and not bool(o.any())


@pytest.mark.parametrize("pooled", [False, True])
def test_packed_forward(host, pooled):
    kw = dict(slots=torch.zeros(2, dtype=torch.int32), s_final=torch.zeros(5, 4, 16, 32)) if pooled else {}
    o, _ = efla.efla_gated_chunk_fwd_varlen(*inputs(9), torch.tensor([1, 3, 6], dtype=torch.int32), **kw)
    assert o.dtype == BF and o.shape == (9, 4, 32) and not bool(o.any())


def test_a_given_output_is_left_alone(host):
    o = torch.full((9, 4, 32), 7.0, dtype=BF)
    got, _ = efla.efla_gated_chunk_fwd_varlen(*inputs(9), torch.tensor([1, 3, 6], dtype=torch.int32), o=o)
    assert got is o and bool((o == 7).all())
    o = torch.full((3, 4, 32), 7.0, dtype=BF)
    got = efla.efla_gated_step(*inputs(3), torch.zeros(7, 4, 16, 32), slots=torch.zeros(3, dtype=torch.int32), o=o)
    assert got is o and bool((o == 7).all())
