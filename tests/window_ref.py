"""The attention over a window with sinks from its definition in 64 bits, each
result with a bound on how far a kernel's may be from it.

The bounds count roundings as tests/cross_ref.py does (u = 2^-24 for a 32-bit
operation, h = finfo(dtype).eps / 2 for a rounding to the I/O type): a score 66 u of
its terms' sizes, a weight the exponent's error and, in bf16, h before its
product, a sum over n terms n u of their sizes, a result h of its own value.
"""
import math

import torch

from cross_ref import U, check, half_step  # noqa: F401  (check: for the tests)


def seen_of(B, Nq, Nk, window=None, sinks=0, q_start=None, kv_len=None, device="cuda"):
    """[B, Nq, Nk]: whether the query attends the key."""
    start = torch.full((B,), Nk - Nq, device=device) if q_start is None else q_start.long()
    n = torch.full((B,), Nk, device=device) if kv_len is None else kv_len.long().clamp(0, Nk)
    p = (start[:, None] + torch.arange(Nq, device=device))[..., None]
    k = torch.arange(Nk, device=device)
    seen = (k <= p) & (p < n[:, None, None])
    return seen if window is None else seen & ((k > p - window) | (k < sinks))


def window(q, k, v, scale, seen, dO=None, o_in=None, weight_step=None):
    """{name: (value, bound)} of O, LSE and, with dO, of dQ, dK, dV; o_in: the
    stored O that the backward is given (its rounding is part of the bound)."""
    dt = q.dtype
    h = half_step(dt)
    hw = (h if dt == torch.bfloat16 else 0.0) if weight_step is None else weight_step
    B, Hq, Nq, _ = q.shape
    Hkv, Nk = k.shape[1:3]
    G = Hq // Hkv
    some, used = seen.any(2)[:, None], seen.any(1)[:, None, :, None]      # queries with keys, keys with queries
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    Q = torch.where(some[..., None], q.double(), zero)
    K = torch.where(used, k.double(), zero).repeat_interleave(G, 1)
    V = torch.where(used, v.double(), zero).repeat_interleave(G, 1)
    s = (scale * (Q @ K.transpose(-1, -2))).masked_fill_(~seen[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    base = torch.where(some.expand_as(lse), lse, zero)
    p = torch.exp(s - base[..., None])
    O = p @ V
    mag = abs(scale) * (Q.abs() @ K.abs().transpose(-1, -2)).amax(-1)      # >= |s|
    ew = U * (66 * mag + 4 * mag + 4 * base.abs() + 8)
    es = ew + U * (Nk + 8)
    out = {}
    A = p @ V.abs()
    out["O"] = (O, 1.05 * (h * O.abs() + (hw + 2 * es)[..., None] * A) + 1e-30)
    out["LSE"] = (torch.where(some.expand_as(lse), lse, torch.full_like(lse, -math.inf)),
                  1.05 * (es + U * (2 * base.abs() + 4)))
    if dO is None:
        return out
    g = torch.where(some[..., None], dO.double(), zero)
    D = (g * O).sum(-1)
    dP = g @ V.transpose(-1, -2)
    dS = p * (dP - D[..., None])
    eP = U * 66 * (g.abs() @ V.abs().transpose(-1, -2))
    stored = (o_in.double() - O).abs() if o_in is not None else h * O.abs()
    eD = (g.abs() * stored).sum(-1) + U * 66 * (g.abs() * O.abs()).sum(-1)
    rel = (hw + ew + U * 2 * base.abs())[..., None]      # the LSE given is rounded to 32 bits
    eS = p * (eP + eD[..., None] + U * (dP.abs() + D.abs()[..., None])) + dS.abs() * rel
    sc = abs(scale)
    fold = lambda x: x.view(B, Hkv, G, *x.shape[2:]).sum(2)  # noqa: E731
    dQ = scale * (dS @ K)
    out["dQ"] = (dQ, 1.05 * (h * dQ.abs() + sc * (eS @ K.abs()) + U * (Nk + 4) * sc * (dS.abs() @ K.abs())) + 1e-30)
    n = U * (G * Nq + 4)
    dK = fold(scale * (dS.transpose(-1, -2) @ Q))
    out["dK"] = (dK, 1.05 * (h * dK.abs() + sc * fold(eS.transpose(-1, -2) @ Q.abs())
                             + n * sc * fold(dS.abs().transpose(-1, -2) @ Q.abs())) + 1e-30)
    dV = fold(p.transpose(-1, -2) @ g)
    out["dV"] = (dV, 1.05 * (h * dV.abs() + fold((p * rel).transpose(-1, -2) @ g.abs())
                             + n * fold(p.transpose(-1, -2) @ g.abs())) + 1e-30)
    return out
