"""The gated entry points and the plan refuse what they cannot run, before
anything is launched (CPU only): the C ABI by status, the binding by ValueError.
And the plain forms that the GPU tests compare with, checked against each other."""
import ctypes

import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _gated as G

BF, F32 = torch.bfloat16, torch.float32
NUL, FAKE, ODD = None, ctypes.c_void_p(4096), ctypes.c_void_p(4098)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


# ------------------------------------------------------------------ C ABI
def fwd(B=1, H=4, Hk=2, L=640, dk=64, dv=64, chunk=64, dt=1, rule=0, ptr=FAKE, q=None, o=None, ws=FAKE, n=1 << 30):
    return efla.lib().efla_gated_chunk_fwd(q or ptr, ptr, ptr, ptr, ptr, NUL, o or ptr, NUL, B, H, Hk, L, dk, dv, chunk, dt,
                                           rule, ws, n, NUL)


def varlen(N=2, P=2, H=4, Hk=2, T=640, dk=64, dv=64, chunk=64, dt=1, rule=0, ptr=FAKE, cu=FAKE, slots=NUL, ws=FAKE, n=1 << 30):
    return efla.lib().efla_gated_chunk_fwd_varlen(ptr, ptr, ptr, ptr, ptr, cu, slots, NUL, N, P, NUL, ptr, NUL, H, Hk, T, dk,
                                                  dv, chunk, dt, rule, ws, n, NUL)


def bwd(B=1, H=4, Hk=2, L=640, dk=64, dv=64, chunk=64, dt=1, rule=0, ptr=FAKE, dq=None, ws=FAKE, n=1 << 30):
    p = ptr
    return efla.lib().efla_gated_chunk_bwd(p, p, p, p, p, NUL, p, NUL, dq or p, p, p, p, p, NUL, B, H, Hk, L, dk, dv, chunk,
                                           dt, rule, ws, n, NUL)


def step(N=2, P=2, H=4, Hk=2, dk=64, dv=64, dt=1, rule=0, ptr=FAKE, state=FAKE, slots=NUL):
    return efla.lib().efla_gated_step(ptr, ptr, ptr, ptr, ptr, state, slots, ptr, N, P, H, Hk, dk, dv, dt, rule, NUL)


def plan(N=2, T=10, chunk=64, lengths=FAKE, cu=FAKE):
    return efla.lib().efla_pack_plan(lengths, NUL, N, T, chunk, cu, NUL, NUL, NUL, NUL)


@pytest.mark.parametrize("call", [fwd, varlen, bwd, step])
def test_shapes_and_enums(call):
    assert call(rule=2) == INVALID and call(rule=-1) == INVALID
    assert call(dt=7) == INVALID
    assert call(H=4, Hk=3) == INVALID and call(Hk=0) == INVALID and call(H=0) == INVALID and call(H=2, Hk=4) == INVALID
    assert call(dk=24) == UNSUPPORTED and call(dv=256) == UNSUPPORTED and call(dk=0) == UNSUPPORTED
    assert call(ptr=NUL) == INVALID


@pytest.mark.parametrize("call", [fwd, varlen, bwd])
def test_chunk_and_workspace(call):
    assert call(chunk=48) == UNSUPPORTED and call(chunk=128) == UNSUPPORTED
    assert call(ws=NUL) == WORKSPACE and call(n=64) == WORKSPACE
    assert call(ws=ODD) == INVALID
    assert call(ptr=ODD) == INVALID  # q, k, v and o move in 16-byte pieces


def test_lengths_and_counts():
    assert fwd(L=-1) == INVALID and fwd(B=0) == INVALID and bwd(L=-1) == INVALID
    assert fwd(q=ODD) == INVALID and fwd(o=ODD) == INVALID and bwd(dq=ODD) == INVALID
    assert varlen(N=-1) == INVALID and varlen(T=-1) == INVALID and varlen(P=-1) == INVALID
    assert varlen(T=1 << 31) == INVALID
    assert varlen(N=3, P=2) == INVALID   # a state per sequence where no slots name them
    assert varlen(cu=NUL) == INVALID
    assert step(N=3, P=2) == INVALID and step(N=-1) == INVALID and step(state=ODD) == INVALID and step(state=NUL) == INVALID
    assert plan(N=-1) == INVALID and plan(T=-1) == INVALID and plan(T=1 << 31) == INVALID
    assert plan(lengths=NUL) == INVALID and plan(cu=NUL) == INVALID
    assert plan(chunk=48) == UNSUPPORTED


def test_nothing_to_do_is_success_without_a_launch():
    assert fwd(L=0, ptr=NUL, ws=NUL, n=0) == OK
    assert bwd(L=0, ptr=NUL, ws=NUL, n=0) == OK
    assert varlen(N=0, P=0, ptr=NUL, cu=NUL, ws=NUL, n=0) == OK
    assert varlen(T=0, ptr=NUL, ws=NUL, n=0) == OK  # and no final states asked for
    assert step(N=0, ptr=NUL, state=NUL) == OK
    # a pool without rows: every row of the batch is without a request
    assert step(P=0, ptr=NUL, state=NUL, slots=FAKE) == OK


def test_workspace_sizes():
    f, v, b = (efla.efla_gated_chunk_fwd_workspace_size, efla.efla_gated_chunk_fwd_varlen_workspace_size,
               efla.efla_gated_chunk_bwd_workspace_size)
    # per chunk of 64: T in fragment order (12 KiB) and the gate block (1 KiB)
    assert f(4, 16, 16, 4096, 128, 128, 64, BF) == 4 * 16 * 64 * 13 * 1024
    assert f(4, 16, 16, 4096, 128, 128, 16, BF) == f(4, 16, 16, 4096, 128, 128, 64, BF)  # whatever chunk is named
    assert f(2, 8, 8, 777, 64, 64, 64, F32) == 0          # fp32: the recurrence needs none
    assert f(1, 16, 8, 10, 128, 128, 64, BF) == 0         # nor does a short sequence
    assert f(1, 4, 3, 640, 64, 64, 64, BF) == 0           # not a shape
    assert v(16, 16, 8, 16384, 128, 128, 64, BF) == 16 * (256 + 16) * 13 * 1024 + 256
    assert b(1, 4, 4, 0, 64, 64, 64, BF) == 0
    for dt in (BF, F32):
        assert b(1, 4, 2, 640, 64, 64, 64, dt) - b(1, 4, 4, 640, 64, 64, 64, dt) == 2 * 640 * 4 * 64 * 4


# ---------------------------------------------------------------- binding
class _NoLaunch:
    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 1 << 20

        def launch(*a):
            raise AssertionError(f"{name} reached the C ABI despite bad arguments")

        return launch


@pytest.fixture
def host(monkeypatch):
    monkeypatch.setattr(efla, "_same", lambda *a: None)
    monkeypatch.setattr(efla, "lib", lambda: _NoLaunch())
    efla._gated_workspace.cache_clear()
    yield
    efla._gated_workspace.cache_clear()


def inputs(lead, H=4, Hk=2, dk=16, dv=32, dt=BF):
    q = torch.zeros(*lead, Hk, dk, dtype=dt)
    return [q, q.clone(), torch.zeros(*lead, H, dv, dtype=dt), torch.zeros(*lead, H, dtype=dt), torch.zeros(*lead, H)]


CALLS = {
    "fwd": ((2, 8), lambda a, **k: efla.efla_gated_chunk_fwd(*a, **k)),
    "bwd": ((2, 8), lambda a, **k: efla.efla_gated_chunk_bwd(*a, k.pop("d_o", torch.zeros_like(a[2])), **k)),
    "varlen": ((9,), lambda a, **k: efla.efla_gated_chunk_fwd_varlen(*a, k.pop("cu", torch.zeros(3, dtype=torch.int32)), **k)),
    "step": ((3,), lambda a, **k: efla.efla_gated_step(*a, k.pop("state", torch.zeros(3, 4, 16, 32)), **k)),
}


@pytest.mark.parametrize("name", CALLS)
def test_binding_rejects_bad_inputs(host, name):
    lead, call = CALLS[name]
    for i in range(5):
        a = inputs(lead)
        a[i] = a[i][..., :-1]          # a wrong last dimension
        if i == 2 and name != "step":
            continue                   # any d_v is a shape to the binding; the library refuses it
        with pytest.raises(ValueError):
            call(a)
        a = inputs(lead)
        a[i] = a[i].to(torch.float64)  # a type of its own
        with pytest.raises(ValueError):
            call(a)
        a = inputs(lead)
        a[i] = a[i][0]                 # a dimension too few
        with pytest.raises(ValueError):
            call(a)
    a = inputs(lead)
    a[4] = a[4].to(BF)                 # g is float32
    with pytest.raises(ValueError):
        call(a)
    with pytest.raises(ValueError):
        call(inputs(lead, H=4, Hk=3))
    with pytest.raises(ValueError):
        call(inputs(lead), rule="midpoint")
    with pytest.raises(ValueError):
        call(inputs(lead, dt=torch.float16))


@pytest.mark.parametrize("name,extra", [
    ("fwd", dict(o=torch.zeros(2, 8, 4, 16, dtype=BF))), ("fwd", dict(o=torch.zeros(2, 8, 4, 32))),
    ("fwd", dict(s0=torch.zeros(2, 4, 32, 16))), ("fwd", dict(s0=torch.zeros(2, 4, 16, 32, dtype=BF))),
    ("fwd", dict(s_final=torch.zeros(1, 4, 16, 32))),
    ("bwd", dict(d_o=torch.zeros(2, 8, 4, 32))), ("bwd", dict(d_o=torch.zeros(2, 8, 4, 16, dtype=BF))),
    ("bwd", dict(ds_final=torch.zeros(2, 4, 16, 31))), ("bwd", dict(s0=torch.zeros(2, 2, 16, 32))),
    ("varlen", dict(cu=torch.zeros(3, dtype=torch.int64))), ("varlen", dict(cu=torch.zeros(1, 3, dtype=torch.int32))),
    ("varlen", dict(s0=torch.zeros(3, 4, 16, 32))),
    ("varlen", dict(slots=torch.zeros(2, dtype=torch.int32))),                                # no pool
    ("varlen", dict(slots=torch.zeros(2, dtype=torch.int32), s0=torch.zeros(5, 4, 16, 32))),  # final states nowhere
    ("varlen", dict(slots=torch.zeros(2, dtype=torch.int32), s0=torch.zeros(5, 4, 16, 32), s_final=torch.zeros(4, 4, 16, 32))),
    ("varlen", dict(slots=torch.zeros(2, dtype=torch.int64), s0=torch.zeros(5, 4, 16, 32), want_final=False)),
    ("varlen", dict(order=torch.zeros(3, dtype=torch.int32))), ("varlen", dict(o=torch.zeros(9, 4, 32))),
    ("step", dict(state=torch.zeros(4, 4, 16, 32))), ("step", dict(state=torch.zeros(3, 4, 32, 16))),
    ("step", dict(state=torch.zeros(3, 4, 16, 32, dtype=BF))), ("step", dict(slots=torch.zeros(2, dtype=torch.int32))),
    ("step", dict(slots=torch.zeros(3, dtype=torch.int64))), ("step", dict(o=torch.zeros(3, 4, 32))),
], ids=lambda x: x if isinstance(x, str) else "-".join(x))
def test_binding_rejects_bad_extras(host, name, extra):
    lead, call = CALLS[name]
    with pytest.raises(ValueError):
        call(inputs(lead), **dict(extra))


def test_plan_binding_rejects(host):
    for bad in (torch.zeros(3, dtype=torch.int64), torch.zeros(1, 3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            efla.efla_pack_plan(bad, 10)
    ln = torch.zeros(3, dtype=torch.int32)
    for kw in (dict(tokens=-1), dict(tokens=2 ** 31), dict(tokens=5, starts=torch.zeros(2, dtype=torch.int32)),
               dict(tokens=5, starts=torch.zeros(3))):
        with pytest.raises(ValueError):
            efla.efla_pack_plan(ln, **kw)


def test_binding_rejects_host_tensors():
    for name, (lead, call) in CALLS.items():
        with pytest.raises(ValueError):
            call(inputs(lead))
    with pytest.raises(ValueError):
        efla.efla_pack_plan(torch.zeros(3, dtype=torch.int32), 10)


# ------------------------------------------------- the plain forms themselves
def chunked(q, k, v, beta, g, S, C, rule):
    """The chunked algebra of csrc/gated.h in float64, one sequence and head."""
    alpha = G.alpha_ref(beta, k, rule)
    o = []
    for a in range(0, len(v), C):
        Q, K, V, al = (x[a:a + C] for x in (q, k, v, alpha))
        Gs = g[a:a + C].cumsum(0)
        gam = torch.exp((Gs[:, None] - Gs[None, :]).tril()).tril()
        A = (al[:, None] * gam * (K @ K.T)).tril(-1)
        T = torch.linalg.inv(torch.eye(len(V), dtype=torch.float64) + A) * al[None, :]
        U = T @ (V - Gs.exp()[:, None] * (K @ S))
        o.append(Gs.exp()[:, None] * (Q @ S) + (gam * (Q @ K.T)) @ U)
        S = Gs[-1].exp() * S + K.T @ ((Gs[-1] - Gs).exp()[:, None] * U)
    return torch.cat(o), S


@pytest.mark.parametrize("rule", ["exact", "euler"])
@pytest.mark.parametrize("C", [1, 7, 16, 64])
def test_chunk_algebra_is_the_recurrence(rule, C):
    x = G.make(1, 50, 1, 1, 8, 6, torch.float64, seed=C)
    a = G.wide(x)
    o, S = G.forward_ref(*a, x["s0"].double(), rule)
    o2, S2 = chunked(*(t[0, :, 0] for t in a), x["s0"].double()[0, 0], C, rule)
    assert G.rel(o2, o[0, :, 0]) < 1e-12 and G.rel(S2, S[0, 0]) < 1e-12


def test_recurrence_without_decay_is_the_oracle():
    import oracle
    x = G.make(2, 20, 3, 3, 5, 4, torch.float64, seed=1)
    x["g"].zero_()
    for rule in ("exact", "euler"):
        o, S = G.forward_ref(*G.wide(x), x["s0"].double(), rule)
        ro, rs = oracle.forward(*(x[n].numpy() for n in ("q", "k", "v", "beta")), x["s0"].double().numpy(), rule=rule)
        assert G.rel(o, torch.from_numpy(ro)) < 1e-12 and G.rel(S, torch.from_numpy(rs)) < 1e-12


def test_gate_gradient_formula():
    """dg by the sum over crossing pairs (csrc/gated_bwd.h) against autograd, one chunk."""
    C, dk, dv = 9, 5, 4
    x = G.make(1, C, 1, 1, dk, dv, torch.float64, seed=4)
    q, k, v, beta, g = (t[0, :, 0].clone().requires_grad_() for t in G.wide(x))
    S = x["s0"].double()[0, 0]
    gen = torch.Generator().manual_seed(3)
    do, dS = torch.randn(C, dv, generator=gen, dtype=torch.float64), torch.randn(dk, dv, generator=gen, dtype=torch.float64)
    o, Sf = chunked(q, k, v, beta, g, S, C, "euler")
    want, = torch.autograd.grad((o * do).sum() + (Sf * dS).sum(), g)
    with torch.no_grad():
        Gs = g.cumsum(0)
        e, w = Gs.exp()[:, None], (Gs[-1] - Gs).exp()[:, None]
        gam = torch.exp((Gs[:, None] - Gs[None, :]).tril()).tril()
        KK = k @ k.T
        A = (beta[:, None] * gam * KK).tril(-1)
        X = torch.linalg.inv(torch.eye(C, dtype=torch.float64) + A)
        T = X * beta[None, :]
        D = v - e * (k @ S)
        U, P = T @ D, gam * (q @ k.T)
        dU = P.T @ do + w * (k @ dS)
        dD, dT, dP0 = T.T @ dU, (dU @ D.T).tril(), (do @ U.T).tril()
        Y1, Y2, Y3 = e * (do @ S.T), w * (U @ dS.T), e * (dD @ S.T)
        dA = -(X.T @ (dT * beta[None, :]) @ X.T).tril(-1)
        M = (dP0 * P).tril(-1) + dA * A
        y = (q * Y1).sum(1) - (k * Y3).sum(1) + M.sum(1) - M.sum(0)
        wj = (k * Y2).sum(1)
        dg = Gs[-1].exp() * (dS * S).sum() + wj.cumsum(0) - wj + y.flip(0).cumsum(0).flip(0)
    assert G.rel(dg, want) < 1e-12


def test_plan_ref():
    cu, order, seq, pos = G.plan_ref([3, 0, -2, 70], 60, [5, 0, 0, 9], 64)
    assert cu == [0, 3, 3, 3, 60] and order == [0, 3, 1, 2]
    assert seq[:4] == [0, 0, 0, 3] and pos[:4] == [5, 6, 7, 9] and seq[-1] == 3
