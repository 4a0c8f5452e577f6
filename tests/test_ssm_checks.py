"""The convolution's, the scan's and the pools' entry points refuse what they cannot
run, before anything is launched (CPU only): the C ABI by status, the binding by
ValueError.  And the plain forms that the GPU tests compare with, checked against
each other."""
import ctypes

import pytest
import torch

from delta_rule_sequence_efla_amd import efla
from tests import _ssm as R

BF, F32 = torch.bfloat16, torch.float32
NUL, FAKE, ODD = None, ctypes.c_void_p(4096), ctypes.c_void_p(4098)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BIG = 1 << 24


# ------------------------------------------------------------------ C ABI
def conv(B=1, L=64, D=64, W=4, silu=1, dt=1, row=64, yrow=None, x=FAKE, p=FAKE, fin=NUL):
    return efla.lib().efla_conv_fwd(x, row, p, NUL, NUL, p, yrow or row, fin, B, L, D, W, silu, dt, NUL)


def conv_varlen(N=2, P=2, T=64, D=64, W=4, silu=1, dt=1, row=64, x=FAKE, p=FAKE, cu=FAKE, slots=NUL, fin=NUL):
    return efla.lib().efla_conv_fwd_varlen(x, row, p, NUL, cu, slots, N, P, NUL, p, row, fin, T, D, W, silu, dt, NUL)


def conv_step(N=2, P=2, D=64, W=4, silu=1, dt=1, row=64, x=FAKE, p=FAKE, slots=NUL):
    return efla.lib().efla_conv_step(x, row, p, NUL, p, slots, p, row, N, P, D, W, silu, dt, NUL)


def conv_bwd(B=1, L=64, D=64, W=4, silu=1, dt=1, row=64, x=FAKE, p=FAKE, dw=FAKE, ws=FAKE, n=1 << 30):
    return efla.lib().efla_conv_bwd(x, row, p, NUL, NUL, p, row, NUL, p, row, dw, NUL, NUL, B, L, D, W, silu, dt, ws, n, NUL)


@pytest.mark.parametrize("call", [conv, conv_varlen, conv_step, conv_bwd])
def test_conv_refusals(call):
    assert call(W=1) == UNSUPPORTED and call(W=5) == UNSUPPORTED and call(D=BIG, row=BIG) == UNSUPPORTED
    assert call(D=0) == INVALID and call(dt=7) == INVALID and call(silu=2) == INVALID
    assert call(row=63) == INVALID and call(row=BIG) == UNSUPPORTED
    assert call(x=NUL) == INVALID and call(p=NUL) == INVALID
    assert call(x=ctypes.c_void_p(4097)) == INVALID and call(x=ODD, dt=0) == INVALID  # not aligned to an element


def test_conv_counts():
    assert conv(B=0) == INVALID and conv(L=-1) == INVALID and conv(yrow=60) == INVALID
    assert conv(L=0, x=NUL, p=NUL) == OK  # and no final state asked for
    assert conv_varlen(N=-1) == INVALID and conv_varlen(T=-1) == INVALID and conv_varlen(T=1 << 31) == INVALID
    assert conv_varlen(P=1) == INVALID and conv_varlen(P=-1, slots=FAKE) == INVALID and conv_varlen(cu=NUL) == INVALID
    assert conv_varlen(N=0, P=0, cu=NUL, x=NUL, p=NUL) == OK and conv_varlen(T=0, x=NUL, p=NUL) == OK
    assert conv_step(P=1) == INVALID and conv_step(N=-1) == INVALID
    assert conv_step(N=0, x=NUL, p=NUL) == OK and conv_step(P=0, slots=FAKE, x=NUL, p=NUL) == OK
    assert conv_bwd(B=0) == INVALID and conv_bwd(L=-1) == INVALID and conv_bwd(dw=NUL) == INVALID
    assert conv_bwd(ws=NUL) == WORKSPACE and conv_bwd(n=64) == WORKSPACE and conv_bwd(ws=ODD) == INVALID
    assert conv(B=1 << 20, L=1 << 20) == UNSUPPORTED and conv_bwd(B=1 << 20, L=1 << 20) == UNSUPPORTED  # 2^32 threads
    size = efla.efla_conv_bwd_workspace_size
    assert size(1, 64, 64, 4) >= 5 * 64 * 4 and size(1, 64, 64, 5) == 0 and size(0, 64, 64, 4) == 0 and size(1, 0, 64, 4) == 0


def ssm_in(p, row, krow=None, dtrow=None):
    return (p, krow or row, p, krow or row, p, row, p, dtrow or row)


def ssm(B=1, H=4, Hk=2, L=640, dk=64, dv=64, dt=1, row=256, p=FAKE, a=FAKE, o=None, krow=None, dtrow=None, orow=None, ws=FAKE,
        n=1 << 34):
    return efla.lib().efla_ssm_fwd(*ssm_in(p, row, krow, dtrow), a, NUL, NUL, NUL, o or p, orow or row, NUL, B, H, Hk, L, dk,
                                   dv, dt, ws, n, NUL)


def ssm_varlen(N=2, P=2, H=4, Hk=2, L=640, dk=64, dv=64, dt=1, row=256, p=FAKE, a=FAKE, o=None, krow=None, dtrow=None,
               cu=FAKE, slots=NUL, ws=FAKE, n=1 << 34):
    return efla.lib().efla_ssm_fwd_varlen(*ssm_in(p, row, krow, dtrow), a, NUL, NUL, cu, slots, NUL, N, P, NUL, o or p, row,
                                          NUL, H, Hk, L, dk, dv, dt, ws, n, NUL)


def ssm_bwd(B=1, H=4, Hk=2, L=640, dk=64, dv=64, dt=1, row=256, p=FAKE, a=FAKE, o=None, krow=None, dtrow=None, ws=FAKE,
            n=1 << 34):
    return efla.lib().efla_ssm_bwd(*ssm_in(p, row, krow, dtrow), a, NUL, NUL, NUL, o or p, row, NUL, p, row, p, row, p, row, p,
                                   row, NUL, NUL, NUL, NUL, B, H, Hk, L, dk, dv, dt, ws, n, NUL)


def ssm_step(N=2, P=2, H=4, Hk=2, dk=64, dv=64, dt=1, row=256, p=FAKE, a=FAKE, krow=None, dtrow=None, state=FAKE, slots=NUL):
    return efla.lib().efla_ssm_step(*ssm_in(p, row, krow, dtrow), a, NUL, NUL, state, slots, p, row, N, P, H, Hk, dk, dv, dt,
                                    NUL)


@pytest.mark.parametrize("call", [ssm, ssm_varlen, ssm_bwd, ssm_step])
def test_ssm_refusals(call):
    assert call(dt=7) == INVALID
    assert call(H=4, Hk=3) == INVALID and call(Hk=0) == INVALID and call(H=0) == INVALID and call(H=2, Hk=4) == INVALID
    assert call(dk=24) == UNSUPPORTED and call(dv=256, row=1024) == UNSUPPORTED and call(dk=0) == UNSUPPORTED
    assert call(row=248) == INVALID and call(krow=120) == INVALID and call(dtrow=3) == INVALID
    assert call(row=BIG) == UNSUPPORTED
    assert call(p=NUL) == INVALID and call(a=NUL) == INVALID


@pytest.mark.parametrize("call", [ssm, ssm_varlen, ssm_bwd])
def test_ssm_alignment(call):
    assert call(p=ODD) == INVALID and call(o=ODD) == INVALID
    assert call(row=260) == INVALID and call(krow=129) == INVALID  # rows that do not start on 16 bytes


def test_ssm_alignment_of_states_and_parameters():
    off, run = ctypes.c_void_p(4104), efla.lib()
    x = ssm_in(FAKE, 256)
    for args in ((off, NUL, NUL, NUL), (NUL, NUL, NUL, off), (NUL, NUL, ctypes.c_void_p(4102), NUL), (NUL, ODD, NUL, NUL)):
        s0, d, bias, sf = args
        assert run.efla_ssm_fwd(*x, FAKE, d, bias, s0, FAKE, 256, sf, 1, 4, 2, 640, 64, 64, 1, FAKE, 1 << 34, NUL) == INVALID
        assert run.efla_ssm_fwd_varlen(*x, FAKE, d, bias, FAKE, NUL, NUL, 2, 2, s0, FAKE, 256, sf, 4, 2, 640, 64, 64, 1, FAKE,
                                       1 << 34, NUL) == INVALID
    for which in range(7):  # s0, ds_final, da, dd, dbias, ds0, ddt
        s0, dsf, da, dd, dbias, ds0, ddt = (((off, off, ODD, ODD, ODD, off, ctypes.c_void_p(4097))[i] if i == which else
                                             (NUL if i < 6 else FAKE)) for i in range(7))
        assert run.efla_ssm_bwd(*x, FAKE, NUL, NUL, s0, FAKE, 256, dsf, FAKE, 256, FAKE, 256, FAKE, 256, ddt, 256, da, dd, dbias,
                                ds0, 1, 4, 2, 640, 64, 64, 1, FAKE, 1 << 34, NUL) == INVALID
    assert ssm_step(p=ctypes.c_void_p(4097)) == INVALID and ssm_step(a=ODD) == INVALID


def test_ssm_workspace_of_cut_sequences():
    size, packed = efla.efla_ssm_fwd_workspace_size, efla.efla_ssm_fwd_varlen_workspace_size
    n = size(1, 4, 4, 3500, 64, 64, BF)  # segments of two chunks of 64 tokens, 28 of them a head
    assert n >= 28 * 4 * (64 * 64 + 1) * 4
    assert size(4, 16, 16, 4096, 128, 128, BF) == 0 and size(1, 4, 4, 300, 64, 64, BF) == 0 and size(1, 4, 3, 3500, 64, 64, BF) == 0
    assert packed(3, 4, 4, 3500, 64, 64, BF) > n and packed(100, 4, 4, 3500, 64, 64, BF) == 0
    assert ssm(L=3500, H=4, Hk=4, ws=NUL, row=256) == WORKSPACE and ssm(L=3500, Hk=4, n=64) == WORKSPACE
    assert ssm(L=3500, Hk=4, ws=ODD) == INVALID and ssm_varlen(L=3500, Hk=4, ws=NUL) == WORKSPACE


def test_ssm_counts():
    assert ssm(B=0) == INVALID and ssm(L=-1) == INVALID and ssm_bwd(B=0) == INVALID and ssm_bwd(L=-1) == INVALID
    assert ssm_varlen(N=-1) == INVALID and ssm_varlen(L=-1) == INVALID and ssm_varlen(L=1 << 31) != OK
    assert ssm_varlen(P=1) == INVALID and ssm_varlen(P=-1, slots=FAKE) == INVALID and ssm_varlen(cu=NUL) == INVALID
    assert ssm_varlen(N=0, P=0, p=NUL, cu=NUL) == OK
    assert ssm(L=0, p=NUL) == OK and ssm_varlen(L=0, p=NUL) == OK  # and no final states asked for
    assert ssm_step(P=1) == INVALID and ssm_step(N=-1) == INVALID and ssm_step(state=ODD) == INVALID
    assert ssm_step(state=NUL) == INVALID and ssm_step(N=0, p=NUL) == OK and ssm_step(P=0, slots=FAKE, p=NUL) == OK
    assert ssm_bwd(ws=NUL) == WORKSPACE and ssm_bwd(n=64) == WORKSPACE and ssm_bwd(ws=ODD) == INVALID
    assert ssm(B=1 << 26) == UNSUPPORTED and ssm_bwd(B=1 << 26) == UNSUPPORTED and ssm_step(N=1 << 26, P=1 << 26) == UNSUPPORTED
    assert efla.efla_ssm_bwd_workspace_size(1, 4, 3, 64, 64, 64, BF) == 0
    assert efla.efla_ssm_bwd_workspace_size(1, 4, 2, 0, 64, 64, BF) == 0


def pools(n=2, P=8, N=3, base=4096, size=64, src=FAKE, dst=FAKE):
    at, sz = (ctypes.c_void_p * max(n, 1))(*[base] * n), (ctypes.c_size_t * max(n, 1))(*[size] * n)
    return efla.lib().efla_pool_copy(at, sz, n, src, dst, N, P, NUL)


def compact(n=2, P=8, N=3, base=4096, size=64, slots=FAKE, new=FAKE, live=FAKE, ws=FAKE, nws=1 << 20):
    at, sz = (ctypes.c_void_p * max(n, 1))(*[base] * n), (ctypes.c_size_t * max(n, 1))(*[size] * n)
    return efla.lib().efla_pool_compact(at, sz, n, slots, N, P, new, live, ws, nws, NUL)


@pytest.mark.parametrize("call", [pools, compact])
def test_pool_refusals(call):
    assert call(n=-1) == INVALID and call(N=-1) == INVALID and call(P=-1) == INVALID
    assert call(base=None) == INVALID and call(base=4097) == INVALID
    assert call(size=0) == INVALID and call(size=7) == INVALID and call(size=1 << 41) == UNSUPPORTED
    assert call(N=1 << 20, size=1 << 30) == UNSUPPORTED  # 2^32 threads
    assert efla.lib().efla_pool_copy(None, None, 1, FAKE, FAKE, 1, 1, NUL) == INVALID


def test_pool_counts():
    assert pools(src=NUL) == INVALID and pools(dst=NUL) == INVALID
    assert pools(N=0, src=NUL) == OK and pools(P=0) == OK and pools(n=0) == OK
    assert compact(slots=NUL) == INVALID and compact(new=NUL) == INVALID and compact(live=NUL) == INVALID
    assert compact(ws=NUL) == WORKSPACE and compact(nws=16) == WORKSPACE and compact(ws=ODD) == INVALID
    assert compact(P=131073) == UNSUPPORTED


# ------------------------------------------------------------------ binding
def test_binding_refuses_shapes_and_places():
    x = R.make_conv(1, 4, 8, 4, BF)
    with pytest.raises(ValueError, match="live on the GPU"):
        efla.efla_conv_fwd(x["x"], x["w"])
    with pytest.raises(ValueError, match="activation"):
        efla.efla_conv_fwd(x["x"], x["w"], activation="relu")
    with pytest.raises(ValueError, match="of one type"):
        efla.efla_conv_fwd(x["x"], x["w"].float())
    with pytest.raises(ValueError, match="of one type"):
        efla.efla_conv_step(x["x"], x["w"], x["s0"])
    s = R.make_scan(1, 4, 4, 2, 16, 16, BF)
    args = [s[n] for n in ("q", "k", "v", "dt", "a")]
    with pytest.raises(ValueError, match="live on the GPU"):
        efla.efla_ssm_fwd(*args)
    with pytest.raises(ValueError, match="multiple"):
        efla.efla_ssm_fwd(s["q"], s["k"], s["v"][:, :, :3], s["dt"][..., :3], s["a"][:3])
    with pytest.raises(ValueError, match="of one type"):
        efla.efla_ssm_fwd(s["q"].float(), *args[1:])
    with pytest.raises(ValueError, match="a must be"):
        efla.efla_ssm_fwd(*args[:4], s["a"].double())
    with pytest.raises(ValueError, match="d must have"):
        efla.efla_ssm_fwd(*args, d=s["d"][:2])
    with pytest.raises(ValueError, match="no pools"):
        efla.efla_pool_copy([], torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="1-D int32"):
        efla.efla_pool_copy([x["s0"]], torch.zeros(1), torch.zeros(1))


def test_rows():
    t = torch.zeros(2, 5, 3, 8)
    assert efla._row(t, 2, "t") == 24 and efla._row(t[0], 1, "t") == 24
    wide = torch.zeros(2, 5, 40)
    assert efla._row(wide[..., 8:32].unflatten(-1, (3, 8)), 2, "t") == 40
    assert efla._row(wide[:, 1, :24].unflatten(-1, (3, 8)), 1, "t") == 200   # one token of each of two requests
    assert efla._row(torch.zeros(1, 1, 3, 8), 2, "t") == 24 and efla._row(torch.zeros(4, 1, 16)[..., :8], 2, "t") == 16
    assert efla._row(torch.zeros(2, 0, 8), 2, "t") == 8
    for bad in (wide.transpose(0, 1)[..., :24], wide[:, ::2, :24], t.transpose(2, 3), wide[..., ::2], t[:1].expand(2, 5, 3, 8)):
        with pytest.raises(ValueError, match="adjacent|evenly"):
            efla._row(bad, 2, "t")


# ------------------------------------------------------------------ plain forms
def test_scan_is_the_gated_recurrence_without_correction():
    x = R.make_scan(1, 20, 2, 1, 8, 8, F32)
    q, k, v, dt, a, d, bias, s0 = R.wide(x)
    o, S = R.scan_ref(q, k, v, dt, a, d, bias, s0)
    delta = torch.nn.functional.softplus(dt + bias)
    T, want = s0.clone(), []
    for t in range(20):
        for h in range(2):
            T[0, h] = torch.exp(a[h] * delta[0, t, h]) * T[0, h] + delta[0, t, h] * torch.outer(k[0, t, 0], v[0, t, h])
        want.append(torch.stack([q[0, t, 0] @ T[0, h] + d[h] * v[0, t, h] for h in range(2)]))
    assert R.rel(o, torch.stack(want)[None]) < 1e-14 and R.rel(S, T) < 1e-14


def test_convolution_is_torchs():
    x = R.make_conv(2, 9, 5, 4, F32, s0=False)
    y, fin = R.conv_ref(x["x"].double(), x["w"].double(), x["bias"].double())
    u = torch.nn.functional.conv1d(torch.nn.functional.pad(x["x"].double().transpose(1, 2), (3, 0)),
                                   x["w"].double()[:, None], x["bias"].double(), groups=5).transpose(1, 2)
    assert R.rel(y, torch.nn.functional.silu(u)) < 1e-14 and torch.equal(fin, x["x"].double()[:, -3:])


def test_scan_gradients_against_differences():
    x = R.make_scan(1, 12, 2, 1, 4, 4, F32)
    gen = torch.Generator().manual_seed(0)
    d_o, dsf = torch.randn(1, 12, 2, 4, generator=gen), torch.randn(1, 2, 4, 4, generator=gen)
    g, _ = R.scan_grads_ref(x, d_o, dsf)
    for name, grad in zip(R.NAMES, R.GRADS):
        way = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        loss = []
        for sign in (1, -1):
            y = {n: x[n].double() + (sign * 1e-6 * way if n == name else 0) for n in x}
            o, S = R.scan_ref(*(y[n] for n in R.NAMES))
            loss.append(float((o * d_o).sum() + (S * dsf).sum()))
        assert abs((loss[0] - loss[1]) / 2e-6 - float((g[grad] * way).sum())) < 1e-7 * float(g[grad].norm() * way.norm() + 1)


def test_compaction():
    assert R.compact_ref([4, 2, -1], 5) == ([1, 0, -1], [(2, 0), (4, 1)], 2)
    assert R.compact_ref([0, 1], 5) == ([0, 1], [], 2)
    assert R.compact_ref([3, 3, 7], 5) == ([0, 0, 7], [(3, 0)], 1)
