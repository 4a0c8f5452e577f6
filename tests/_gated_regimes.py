"""Inputs of the gated delta rule in regimes of their own: states that outlive a
chunk of 64 tokens many times over, and keys far from unit length; and the chunk
algebra in 64 bits with its carry left out, to show that the first of them see it."""
import math

import torch

from tests import _gated as G


def slow(B, L, H, Hk, dk, dv, dtype, seed, lead=None):
    """Heads of slow decay: the first none at all, the others -d exp(N(0, 0.5)) a token with d from
    0.001 to 0.01, so that a chunk of 64 leaves between half of a state and all of it."""
    x = G.make(B, L, H, Hk, dk, dv, dtype, seed=seed, lead=lead)
    gen = torch.Generator().manual_seed(seed + 500)
    d = torch.exp(torch.linspace(math.log(1e-3), math.log(1e-2), H))
    d[0] = 0.0
    x["g"] = (-d * torch.exp(0.5 * torch.randn(x["g"].shape, generator=gen))).float()
    return x


def stiff(B, L, H, Hk, dk, dv, dtype, seed, lam):
    """Keys of squared length lam ("spread": log-uniform from 0.1 to 1000 by token), every fifth of them zero; slow
    heads as above."""
    x = slow(B, L, H, Hk, dk, dv, dtype, seed)
    gen = torch.Generator().manual_seed(seed + 900)
    shape = (*x["k"].shape[:-1], 1)
    sq = torch.full(shape, float(lam)) if lam != "spread" else 0.1 * 10.0 ** (4.0 * torch.rand(shape, generator=gen))
    k = x["k"].double()
    k = k / k.norm(dim=-1, keepdim=True) * sq.sqrt().double()
    k[:, 2::5] = 0.0
    x["k"] = k.to(dtype)
    return x


def chunked(q, k, v, beta, g, S, rule, carry=True, C=64):
    """[B, L, Hk or H, *] in 64 bits, chunk by chunk; carry=False: the factor e^{G_C} of the state before a full
    chunk taken as zero.  -> (o, S)."""
    r = v.shape[2] // k.shape[2]
    q, k = (t.repeat_interleave(r, dim=2) for t in (q, k))
    alpha = G.alpha_ref(beta, k, rule)
    q, k, v, alpha, g = (t.movedim(2, 1) for t in (q, k, v, alpha, g))
    L, os = v.shape[2], []
    for a in range(0, L, C):
        Q, K, V, al, gg = (t[:, :, a:a + C] for t in (q, k, v, alpha, g))
        n = V.shape[2]
        Gs = gg.cumsum(-1)
        e, w = Gs.exp().unsqueeze(-1), (Gs[..., -1:] - Gs).exp().unsqueeze(-1)
        gam = (Gs.unsqueeze(-1) - Gs.unsqueeze(-2)).tril().exp().tril()
        A = (al.unsqueeze(-1) * gam * (K @ K.transpose(-1, -2))).tril(-1)
        U = torch.linalg.solve_triangular(A + torch.eye(n, dtype=A.dtype), al.unsqueeze(-1) * (V - e * (K @ S)), upper=False)
        os.append(e * (Q @ S) + (gam * (Q @ K.transpose(-1, -2))) @ U)
        end = e[:, :, -1:] if carry or n < C else torch.zeros_like(e[:, :, -1:])
        S = end * S + K.transpose(-1, -2) @ (w * U)
    return torch.cat(os, 2).movedim(1, 2), S
