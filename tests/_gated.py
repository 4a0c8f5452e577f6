"""Plain forms of the gated delta rule and of a packed batch's plan, in 64 bits,
token by token, and the tolerances the kernels are held to.

Errors are relative in the 2-norm per tensor, ||x - y|| / ||y||.

Float32 inputs.  A token's update rounds a sum of d_k products and about eight
further values; the update does not expand the state (decays <= 1, 0 <= alpha
|k|^2 <= 1), so errors of independent sign add up to sqrt(L (d_k + 8)) 2^-24 of
its norm after L tokens; FACTOR allows four times that, and 16 for gradients,
whose sums run over d_v and the chunk as well.

bf16 inputs (exact products, float32 sums).  A rounding to bf16 is off by at
most 2^-8.  o: the state, P and U as operands, and o itself, four roundings.
Gradients: on the longest path five (the state or its gradient, D or dU, U or
dD, dP, the gradient itself).  States: float32 operands go in as two bf16 parts
(2^-16 each at most): S, D, T and U per chunk and the dropped low-by-low
product, five in all, independent from chunk to chunk.
"""
import math

import torch

FACTOR = {"out": 4, "grad": 16}


def tol32(L, dk, what="out"):
    return FACTOR[what] * 2.0 ** -24 * math.sqrt(max(L, 1) * (dk + 8))


def tol_o(dtype, L, dk):
    return tol32(L, dk) if dtype == torch.float32 else 4 * 2.0 ** -8


def tol_s(dtype, L, dk):
    two_parts = 0.0 if dtype == torch.float32 else 5 * 2.0 ** -16 * math.sqrt(max(1, -(-L // 16)))
    return tol32(L, dk) + two_parts


def tol_grad(dtype, L, dk):
    return tol32(L, dk, "grad") if dtype == torch.float32 else 5 * 2.0 ** -8


def rel(x, y) -> float:
    x, y = x.detach().double().cpu(), y.detach().double().cpu()
    assert x.shape == y.shape, (x.shape, y.shape)
    n = float(y.norm())
    d = float((x - y).norm())
    return d / n if n else d


def alpha_ref(beta, k, rule):
    if rule == "euler":
        return beta
    lam = (k * k).sum(-1)
    x = beta * lam
    small = x.abs() < 1e-9
    safe = torch.where(small, torch.ones_like(lam), lam)
    return torch.where(small, beta, -torch.expm1(-x) / safe)


def forward_ref(q, k, v, beta, g, s0=None, rule="exact"):
    """[B, L, Hk or H, *] in float64 -> (o, S)."""
    B, L, H, dv = v.shape
    r = H // k.shape[2]
    q, k = (x.repeat_interleave(r, dim=2) for x in (q, k))
    S = torch.zeros(B, H, k.shape[-1], dv, dtype=torch.float64, device=v.device) if s0 is None else s0
    alpha = alpha_ref(beta, k, rule)
    os = []
    for t in range(L):
        S = torch.exp(g[:, t])[..., None, None] * S
        u = alpha[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        os.append((S * q[:, t, :, :, None]).sum(-2))
    o = torch.stack(os, 1) if os else torch.zeros_like(v)
    return o, S


def make(B, L, H, Hk, dk, dv, dtype, seed=0, decay=0.3, s0=True, lead=None):
    """Inputs on the CPU in `dtype` (g and s0 float32): unit-norm keys scaled by U[0.7, 1.2]."""
    gen = torch.Generator().manual_seed(seed)
    lead = (B, L) if lead is None else lead

    def n(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    k = n(*lead, Hk, dk)
    k = k / k.norm(dim=-1, keepdim=True) * (0.7 + 0.5 * torch.rand(*lead, Hk, 1, generator=gen, dtype=torch.float64))
    x = {"q": n(*lead, Hk, dk) * dk ** -0.5, "k": k, "v": n(*lead, H, dv), "beta": torch.sigmoid(n(*lead, H))}
    x = {a: b.to(dtype) for a, b in x.items()}
    x["g"] = (-decay * n(*lead, H).exp()).float()
    x["s0"] = (0.3 * n(B, H, dk, dv)).float() if s0 else None
    return x


NAMES = ("q", "k", "v", "beta", "g")


def wide(x):
    return [x[n].double() for n in NAMES]


def plan_ref(lengths, T, starts=None, chunk=64):
    lengths = [max(int(x), 0) for x in lengths]
    starts = [0] * len(lengths) if starts is None else [int(x) for x in starts]
    cu = [0]
    for x in lengths:
        cu.append(min(cu[-1] + x, T))
    n = [-(-(b - a) // chunk) for a, b in zip(cu, cu[1:])]
    order = sorted(range(len(lengths)), key=lambda u: (-n[u], u)) if len(lengths) <= 4096 else list(range(len(lengths)))
    seq, pos = [-1] * T, [-1] * T
    for u, (a, b) in enumerate(zip(cu, cu[1:])):
        for t in range(a, b):
            seq[t], pos[t] = u, t - a + starts[u]
    return cu, order, seq, pos
