"""Plain forms of the selective state space scan, of the short causal convolution
and of the moves of pool rows, in 64 bits, and the tolerances the kernels are
held to.

Errors are relative in the 2-norm per tensor, ||x - y|| / ||y||; a rounding to
bf16 is off by at most 2^-8 of the value, to float32 by 2^-24.

Convolution.  y is a sum of at most 5 products and a SiLU of about 6 operations
in float32, whose exponential is taken of a float32 product (off by |u| 2^-24,
|u| < 16 here): 32 * 2^-24, then one rounding to the output's type.  Gradients of
weights and bias sum n terms of independent errors: the bound of a term times the
ratio of the terms' absolute sum to the result is taken in full, with
sqrt(n) 2^-24 for the summation.

Scan, float32.  After L tokens the errors of independent sign in sums of d_k
products and about eight further roundings add up to sqrt(L (d_k + 8)) 2^-24 of
the state's norm (decays <= 1 do not expand it); 4 times that is allowed, 16 for
gradients, whose sums run over d_v and the chunk as well.

Scan, bf16.  o: P, the state as an operand and o itself, three roundings of 2^-8.
States and ds0: each float32 operand as three bf16 parts, off by 2^-24, which the
float32 bound covers.  dq, dk, dv: the longest path rounds the
state (or its gradient) or P (or dP), and the result: three.  ddt: one rounding of
the result.  da, dbias, dd: sums over all tokens of float32
terms, held to the sum of the terms' absolute values.
"""
import math

import torch

BF, F32 = torch.bfloat16, torch.float32


def rel(x, y, scale=None) -> float:
    x, y = x.detach().double().cpu(), y.detach().double().cpu()
    assert x.shape == y.shape, (x.shape, y.shape)
    n = float((y if scale is None else scale.double().cpu()).norm())
    d = float((x - y).norm())
    return d / n if n else d


def step_of(dtype):
    return torch.finfo(dtype).eps / 2


def tol_conv(dtype):
    return 32 * 2.0 ** -24 + (step_of(dtype) if dtype == BF else 0.0)


def tol32(L, dk, what="out"):
    return {"out": 4, "grad": 16}[what] * 2.0 ** -24 * math.sqrt(max(L, 1) * (dk + 8))


def tol_o(dtype, L, dk):
    return tol32(L, dk) + (3 * 2.0 ** -8 if dtype == BF else 0.0)


def tol_s(dtype, L, dk):
    return tol32(L, dk)


def tol_grad(dtype, L, dk, name):
    rounded = {"dq": 3 * 2.0 ** -8, "dk": 3 * 2.0 ** -8, "dv": 3 * 2.0 ** -8, "ddt": 2.0 ** -8}
    return tol32(L, dk, "grad") + (rounded.get(name, 0.0) if dtype == BF else 0.0)


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def scan_ref(q, k, v, dt, a, d=None, bias=None, s0=None):
    """[B, L, Hk or H, *] in float64, token by token -> (o, S)."""
    B, L, H, dv = v.shape
    r = H // k.shape[2]
    q, k = (x.repeat_interleave(r, dim=2) for x in (q, k))
    S = torch.zeros(B, H, k.shape[-1], dv, dtype=torch.float64, device=v.device) if s0 is None else s0
    delta = softplus(dt if bias is None else dt + bias)
    os = []
    for t in range(L):
        S = torch.exp(a * delta[:, t])[..., None, None] * S
        S = S + (delta[:, t, :, None] * k[:, t])[..., None] * v[:, t, :, None, :]
        o = (S * q[:, t, :, :, None]).sum(-2)
        os.append(o if d is None else o + d[:, None] * v[:, t])
    return (torch.stack(os, 1) if os else torch.zeros_like(v)), S


def make_scan(B, L, H, Hk, dk, dv, dtype, seed=0, s0=True, lead=None, extras=True, steps=(0.001, 0.1)):
    """Inputs on the CPU in `dtype` (a, d, bias, s0 float32), as a layer makes them."""
    gen = torch.Generator().manual_seed(seed)
    lead = (B, L) if lead is None else lead

    def n(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    x = {"q": n(*lead, Hk, dk) * dk ** -0.5, "k": n(*lead, Hk, dk) * dk ** -0.5, "v": n(*lead, H, dv), "dt": n(*lead, H)}
    x = {name: t.to(dtype) for name, t in x.items()}
    x["a"] = -(1 + 15 * torch.rand(H, generator=gen)).float()
    step = torch.exp(torch.rand(H, generator=gen, dtype=torch.float64) * math.log(steps[1] / steps[0]) + math.log(steps[0]))
    x["d"] = n(H).float() if extras else None
    x["bias"] = torch.log(torch.expm1(step)).float() if extras else None
    x["s0"] = (0.3 * n(B, H, dk, dv)).float() if s0 else None
    return x


NAMES = ("q", "k", "v", "dt", "a", "d", "bias", "s0")
GRADS = ("dq", "dk", "dv", "ddt", "da", "dd", "dbias", "ds0")


def wide(x):
    return [None if x[n] is None else x[n].double() for n in NAMES]


def scan_grads_ref(x, d_o, ds_final=None):
    """Gradients by autograd through scan_ref, and the absolute sums of the terms of da, dd and dbias."""
    ins = [None if t is None else t.clone().requires_grad_() for t in wide(x)]
    L = x["v"].shape[1]
    # a, d and bias once a token, so that the terms of their sums are seen
    per = [None if t is None else t.detach().expand(x["dt"].shape).clone().requires_grad_() for t in ins[4:7]]
    q, k, v, dt = ins[:4]
    B, _, H, dv = v.shape
    r = H // k.shape[2]
    qq, kk = (t.repeat_interleave(r, dim=2) for t in (q, k))
    S = torch.zeros(B, H, k.shape[-1], dv, dtype=torch.float64) if ins[7] is None else ins[7]
    delta = softplus(dt if per[2] is None else dt + per[2])
    loss = 0.0
    for t in range(L):
        S = torch.exp(per[0][:, t] * delta[:, t])[..., None, None] * S
        S = S + (delta[:, t, :, None] * kk[:, t])[..., None] * v[:, t, :, None, :]
        o = (S * qq[:, t, :, :, None]).sum(-2)
        o = o if per[1] is None else o + per[1][:, t, :, None] * v[:, t]
        loss = loss + (o * d_o[:, t].double()).sum()
    if ds_final is not None:
        loss = loss + (S * ds_final.double()).sum()
    want = [t for t in (*ins[:4], *per, ins[7]) if t is not None]
    got = list(torch.autograd.grad(loss, want, allow_unused=True))
    got = [torch.zeros_like(t) if y is None else y for t, y in zip(want, got)]
    g, scale = {}, {}
    for name, t in zip(GRADS, (*ins[:4], *per, ins[7])):
        if t is None:
            g[name] = None
            continue
        y = got.pop(0)
        if name in ("da", "dd", "dbias"):
            g[name], scale[name] = y.sum((0, 1)), y.abs().sum((0, 1))
        else:
            g[name] = y
    return g, scale


def conv_ref(x, w, bias=None, s0=None, silu=True):
    """x [B, L, D] in float64 -> (y, the last W - 1 inputs)."""
    W = w.shape[1]
    s0 = x.new_zeros(x.shape[0], W - 1, x.shape[2]) if s0 is None else s0
    full = torch.cat([s0, x], 1)
    u = torch.zeros_like(x) if bias is None else bias.expand(x.shape)
    for i in range(W):
        u = u + w[:, i] * full[:, i:i + x.shape[1]]
    return (u / (1 + torch.exp(-u)) if silu else u), full[:, x.shape[1]:]


def make_conv(B, L, D, W, dtype, seed=0, s0=True, bias=True, lead=None):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    lead = (B, L) if lead is None else lead
    return {"x": n(*lead, D).to(dtype), "w": (0.5 * n(D, W)).to(dtype), "bias": (0.5 * n(D)).to(dtype) if bias else None,
            "s0": n(B, W - 1, D).to(dtype) if s0 else None}


def compact_ref(slots, P):
    """New rows and the moves (from, to) of a compaction, from Python lists."""
    used = sorted({s for s in slots if 0 <= s < P})
    K = len(used)
    late = [s for s in used if s >= K]
    holes = [r for r in range(K) if r not in used]
    to = dict(zip(late, holes))
    return [to.get(s, s) for s in slots], list(to.items()), K


def in_wider_rows(t, lead, extra, gen=None):
    """A copy of t whose tokens' rows are `extra` elements longer than their values."""
    flat = t.flatten(lead)
    rows = torch.full((*t.shape[:lead], flat.shape[-1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    rows[..., :flat.shape[-1]] = flat
    return rows[..., :flat.shape[-1]].unflatten(-1, t.shape[lead:])


def rate_gradient_ref(x, d_o):
    """da of a scan from no state in float64, and the root of the summed squares of the terms that its rounding errors
    scale: over all pairs i > j of every head, with T_ij = (dO_i . v_j) (q_i . k_j) e^{G_i - G_j} D_j,
    (D_{j+1} + .. + D_i) T_ij, the dot product dO_i . v_j by the norm of its terms."""
    q, k, v, dt, a, d, bias, _ = wide(x)
    r = v.shape[2] // k.shape[2]
    q, k = (t.repeat_interleave(r, 2).transpose(1, 2) for t in (q, k))  # [B, H, L, *]
    v, w = v.transpose(1, 2), d_o.double().transpose(1, 2)
    D = softplus(dt + (0 if bias is None else bias)).transpose(1, 2)
    C = D.cumsum(-1)
    apart = (C[..., :, None] - C[..., None, :]).tril(-1)
    f = torch.exp(a[:, None, None] * apart).tril(-1) * D[..., None, :] * (q @ k.transpose(-1, -2)) * apart
    da = (f * (w @ v.transpose(-1, -2))).sum((0, 2, 3))
    return da, (f * f * ((w * w) @ (v * v).transpose(-1, -2))).sum((0, 2, 3)).sqrt()
