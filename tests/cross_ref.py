"""The cross attention and the query/key norm from their definitions in 64
bits, each result with a bound on how far a kernel's may be from it.

The bounds count roundings (u = 2^-24 for a 32-bit operation, h =
finfo(dtype).eps / 2 for a rounding to the I/O type, to first order, times
1.05 for the products of several):
  score      64-term products summed in 32 bits, scaled: <= 66 u scale sum_d |q_d k_d|
  weight p   relative: that of the exponent (the score and its maximum or
             LSE, each also rounded once at its own size) + 2^-22 of the exponential,
             and h where a kernel rounds weights before a product (bf16)
  sums       over n terms: n u of the sum of magnitudes
  result     h of its own value
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def keep_of(B, Nk, kv_len=None, key_mask=None, device="cpu"):
    keep = torch.ones(B, Nk, dtype=torch.bool, device=device)
    if kv_len is not None:
        keep &= torch.arange(Nk, device=device)[None] < kv_len.long().clamp(0, Nk)[:, None]
    if key_mask is not None:
        keep &= key_mask.bool()
    return keep


def cross(q, k, v, scale, kv_len=None, key_mask=None, dO=None, o_in=None):
    """{name: (value, bound)} of O, LSE and, with dO, of dQ, dK, dV; o_in: the
    stored O that the backward is given (its rounding is part of the bound)."""
    dt = q.dtype
    h = half_step(dt)
    hw = h if dt == torch.bfloat16 else 0.0
    B, Hq, Nq, _ = q.shape
    Hkv, Nk = k.shape[1:3]
    G = Hq // Hkv
    keep = keep_of(B, Nk, kv_len, key_mask, q.device)[:, None, None]
    clean = keep.transpose(-1, -2)
    Q = q.double()
    K = torch.where(clean, k.double(), torch.zeros((), dtype=torch.float64, device=q.device)).repeat_interleave(G, 1)
    V = torch.where(clean, v.double(), torch.zeros((), dtype=torch.float64, device=q.device)).repeat_interleave(G, 1)
    s = (scale * (Q @ K.transpose(-1, -2))).masked_fill(~keep, -math.inf)
    some = keep.any(-1)
    lse = torch.logsumexp(s, -1)
    base = torch.where(some.expand_as(lse), lse, torch.zeros_like(lse))
    p = torch.exp(s - base[..., None])
    O = p @ V
    # relative bound of a weight, per row (the largest score error of the row)
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
    g = dO.double()
    D = (g * O).sum(-1)
    dP = g @ V.transpose(-1, -2)
    dS = p * (dP - D[..., None])
    eP = U * 66 * (g.abs() @ V.abs().transpose(-1, -2))
    stored = (o_in.double() - O).abs() if o_in is not None else h * O.abs()
    eD = (g.abs() * stored).sum(-1) + U * 66 * (g.abs() * O.abs()).sum(-1)
    # the LSE given is rounded to 32 bits
    rel = (hw + ew + U * 2 * base.abs())[..., None]
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


def qk_norm(x, heads, wq, wk, eps, rotary=None, positions=None, interleaved=False, grads=None):
    """{name: (value, bound)} of Q, K, V or, with grads = (dQ, dK, dV), of dx, dwq, dwk."""
    dt = x.dtype
    h = half_step(dt)
    B, N, _ = x.shape
    Hq, Hk, Hv = heads
    X = x.double().view(B, N, Hq + Hk + Hv, 64)
    dev = x.device
    cos = torch.ones(B, N, 1, 32, dtype=torch.float64, device=dev)
    sin = torch.zeros_like(cos)
    half = 0
    if rotary is not None:
        half = rotary[0].shape[1]
        pos = torch.arange(N, device=dev) if positions is None else positions.long()
        pos = pos.expand(B, N)
        ok = (pos >= 0) & (pos < rotary[0].shape[0])
        for t, tab in ((cos, rotary[0]), (sin, rotary[1])):
            t[..., 0, :half][ok] = tab.double()[pos[ok]]
    i = torch.arange(half, device=dev)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[..., :half], sin[..., :half]

    def turn(y, back=False, size=False):
        z = y.clone()
        t = -s if back else s
        if size:   # sums of magnitudes
            z[..., a], z[..., b] = (y[..., a] * c.abs() + y[..., b] * s.abs(), y[..., a] * s.abs() + y[..., b] * c.abs())
        else:
            z[..., a], z[..., b] = y[..., a] * c - y[..., b] * t, y[..., a] * t + y[..., b] * c
        return z

    out = {}
    parts = {"q": (X[:, :, :Hq], wq), "k": (X[:, :, Hq:Hq + Hk], wk)}
    dxs, dxe = [], []
    for j, (name, (xx, w)) in enumerate(parts.items()):
        W = torch.ones(64, dtype=torch.float64, device=dev) if w is None else w.double()
        r = torch.ones_like(xx[..., :1]) if w is None else (xx.square().mean(-1, keepdim=True) + eps).rsqrt()
        n = xx * r
        if grads is None:
            y = n * W
            z = turn(y)
            # r: 8 terms a lane, 3 joins, mean, eps, rsqrt (2 ulp): 16 u; products and the rotation 6 u
            e = 1.05 * (h * z.abs() + 24 * U * turn(y.abs(), size=True)) + 1e-30
            out[name.upper()] = (z.transpose(1, 2), e.transpose(1, 2))
        else:
            dz = grads[j].double().transpose(1, 2) if (Hq, Hk)[j] else torch.zeros_like(xx)
            dy, ay = turn(dz, back=True), turn(dz.abs(), size=True)
            if w is not None:
                dw = (dy * n).sum((0, 1, 2))
                rows = B * N * xx.shape[2]
                out["dw" + name] = (dw, 1.05 * (h * dw.abs() + U * (rows + 32) * (ay * n.abs()).sum((0, 1, 2))) + 1e-30)
            g, ag = dy * W, ay * W.abs()
            if w is None:
                dx, size = g, ag
            else:
                dx = r * (g - n * (g * n).mean(-1, keepdim=True))
                size = r * (ag + n.abs() * (ag * n.abs()).mean(-1, keepdim=True))
            dxs.append(dx)
            dxe.append(1.05 * (h * dx.abs() + 64 * U * size) + 1e-30)
    if grads is None:
        vv = X[:, :, Hq + Hk:].transpose(1, 2)
        out["V"] = (vv, torch.zeros_like(vv))
        return out
    dvv = grads[2].double().transpose(1, 2) if Hv else X[:, :, Hq + Hk:]
    out["dx"] = (torch.cat([*dxs, dvv], 2).reshape(B, N, -1),
                 torch.cat([*dxe, torch.zeros_like(dvv)], 2).reshape(B, N, -1))
    return out


def check(name, got, want):
    """got within the bound of want = (value, bound), infinities equal."""
    value, bound = want
    got = got.double()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    inf = torch.isinf(value)
    assert torch.equal(got[inf], value[inf]), f"{name}: infinities differ"
    d = (got - value).abs()
    d[inf] = 0.0
    bad = ~(d <= bound)
    bad[inf] = False
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {d.numel()} values outside their bounds, first at {at}: "
                             f"{float(got[at])!r} for {float(value[at])!r}, bound {float(bound[at]):.3g}")
