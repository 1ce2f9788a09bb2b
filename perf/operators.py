"""The query/key norm with position rotation and the cross attention: their
plain forms, their calls, and the cases they are measured on.

A case is a dict of plain values:

  op       "norm_fwd", "norm_bwd": RMS norm of every query and key head and
           the position rotation, from the packed projection [B, N, (Hq + Hk +
           Hv) 64] to Q, K, V [B, H, N, 64], and its gradient
           "cross_fwd", "cross_bwd": attention of Nq queries to Nk states,
           and its gradient
  dtype    "bf16" or "f32", the type of every tensor but the statistics
  mask     what a sequence attends: "none" (all states), "len" (its own
           length, one sequence without any where there are at least four),
           "mask" (a truth value for each state, three of four kept)
"""
import math

import torch

own = False

HEAD = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _norm(name, op, dtype, B, N, Hq, Hk, rot, pairs, cls):
    c = {"op": op, "dtype": dtype, "B": B, "N": N, "Hq": Hq, "Hk": Hk, "rot": rot, "pairs": pairs, "cls": cls}
    return {"name": name, **c} if name else c


def _cross(name, op, dtype, B, Hq, Hkv, Nq, Nk, mask):
    c = {"op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "mask": mask}
    return {"name": name, **c} if name else c


def listed():
    return [
        # an encoder block on 14 x 14 patches and a class token, which is not rotated
        _norm("norm_fwd_vitb", "norm_fwd", "bf16", 64, 197, 12, 12, 64, "halves", True),
        # one new token of each of eight sequences, four query heads to a key head
        _norm("norm_fwd_token", "norm_fwd", "bf16", 8, 1, 16, 4, 64, "halves", False),
        # the same block's training step
        _norm("norm_bwd_train", "norm_bwd", "bf16", 256, 197, 12, 12, 64, "halves", True),
        # 128 x 128 patches in 32 bits, half of each head rotated, neighbours paired
        _norm("norm_bwd_long_f32", "norm_bwd", "f32", 2, 16385, 16, 16, 32, "neighbours", True),
        # one token of four decoders against an image's states
        _cross("cross_fwd_token_image", "cross_fwd", "bf16", 4, 12, 12, 1, 197, "none"),
        # one token of sixteen decoders against states of a 128 x 128 image, of several lengths
        _cross("cross_fwd_token_long", "cross_fwd", "bf16", 16, 16, 4, 1, 16385, "len"),
        # a decoder's queries against the patches that a masked encoder kept
        _cross("cross_fwd_masked", "cross_fwd", "bf16", 64, 12, 12, 65, 197, "mask"),
        # queries of one image against the states of a video clip, padded to the longest
        _cross("cross_fwd_video", "cross_fwd", "bf16", 8, 12, 12, 197, 1569, "len"),
        # queries of a clip against a 128 x 128 image
        _cross("cross_fwd_long", "cross_fwd", "bf16", 2, 16, 16, 1569, 16385, "none"),
        # training: image queries, clip states, three query heads to a key head
        _cross("cross_bwd_video", "cross_bwd", "bf16", 8, 12, 4, 197, 1569, "len"),
        # training: clip queries, image states
        _cross("cross_bwd_long", "cross_bwd", "bf16", 2, 16, 16, 1569, 16385, "none"),
        # training in 32 bits on masked patches
        _cross("cross_bwd_f32", "cross_bwd", "f32", 4, 12, 12, 197, 197, "mask"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.3:
        op = rng.choice(["norm_fwd", "norm_bwd"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        Hk = rng.choice([1, 3, 4, 12, 16])
        Hq = Hk * rng.choice([1, 1, 3, 4])
        while True:
            B, N = _spread(rng, 1, 64), _spread(rng, 1, 16385)
            if B * N * (Hq + 2 * Hk) <= 2 * 16385 * 48:
                break
        return _norm(None, op, dtype, B, N, Hq, Hk, rng.choice([16, 32, 64, 64]), rng.choice(["halves", "neighbours"]),
                     N > 1 and rng.random() < 0.5)
    op = rng.choice(["cross_fwd", "cross_fwd", "cross_bwd", "cross_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    # all of the largest listed case for 16 bits; the 32-bit path is for smaller models
    most = 2 * 16 * 1569 * 16385 if dtype == "bf16" else 2 * 16 * 1569 * 197
    Hkv = rng.choice([1, 3, 4, 12, 16])
    Hq = Hkv * rng.choice([1, 1, 1, 2, 3, 4])
    while True:
        B = _spread(rng, 1, 64)
        Nq = 1 if op == "cross_fwd" and rng.random() < 0.25 else _spread(rng, 1, 2048)
        # the gradients of queries and keys of a single state are zeros: from three on there are others
        Nk = _spread(rng, 1 if op == "cross_fwd" else 3, 16385)
        if B * Hq * Nq * Nk <= most and B * Hkv * Nk <= 16 * 4 * 16385:
            break
    return _cross(None, op, dtype, B, Hq, Hkv, Nq, Nk, rng.choice(["none", "len", "len", "mask"]))


# ------------------------------------------------------------------- inputs

def _lengths(case):
    """Lengths of the sequences, the same for every seed but for their order."""
    B, Nk = case["B"], case["Nk"]
    lens = [max(1, round(Nk * (1.0 - 0.5 * i / max(1, B - 1)))) for i in range(B)]
    if B >= 4:
        lens[-1] = 0   # a sequence whose states were all dropped
    return lens


def _kept(case):
    """States that a masked sequence attends."""
    return max(1, (3 * case["Nk"]) // 4)


def _table(case, dev):
    """cos and sin of each position's angles, [positions, rot / 2], from 64 bits."""
    n, half = max(1, case["N"]), case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
    ang = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * freq[None]
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = TYPES[case["dtype"]]

    def randn(*shape, dtype=t):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    B = case["B"]
    s = {"case": case}
    if case["op"].startswith("norm"):
        N, Hq, Hk = case["N"], case["Hq"], case["Hk"]
        s["x"] = randn(B, N, (Hq + 2 * Hk) * HEAD)
        s["wq"] = (1.0 + 0.1 * randn(HEAD, dtype=torch.float32)).to(t)
        s["wk"] = (1.0 + 0.1 * randn(HEAD, dtype=torch.float32)).to(t)
        s["cos"], s["sin"] = _table(case, dev)
        if N == 1:    # one token each: the sequences are at places of their own
            s["cos"], s["sin"] = _table({**case, "N": 16385}, dev)
            s["pos"] = torch.randint(0, 16385, (B, 1), generator=g, device=dev, dtype=torch.int32)
        else:
            s["pos"] = torch.arange(N, device=dev, dtype=torch.int32) - (1 if case["cls"] else 0)
        if case["op"] == "norm_bwd":
            s["dq"], s["dk"], s["dv"] = randn(B, Hq, N, HEAD), randn(B, Hk, N, HEAD), randn(B, Hk, N, HEAD)
        return s
    Hq, Hkv, Nq, Nk = case["Hq"], case["Hkv"], case["Nq"], case["Nk"]
    # as the projections leave them: queries [B, N, H, 64], keys and values side by side
    s["q"] = randn(B, Nq, Hq, HEAD).transpose(1, 2)
    kv = randn(B, Nk, 2, Hkv, HEAD)
    s["k"], s["v"] = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    s["scale"] = HEAD ** -0.5
    s["len"] = s["mask"] = None
    if case["mask"] == "len":
        order = torch.randperm(B, generator=g, device=dev)
        s["len"] = torch.tensor(_lengths(case), device=dev, dtype=torch.int32)[order].contiguous()
    elif case["mask"] == "mask":
        rank = torch.rand(B, Nk, generator=g, device=dev).argsort(1).argsort(1)
        s["mask"] = rank < _kept(case)
    if case["op"] == "cross_bwd":
        s["do"] = randn(B, Nq, Hq, HEAD).transpose(1, 2)
        s["o"], s["lse"] = _plain_cross_fwd(s)
    return s


# --------------------------------------------------------------- plain forms

def _rotate(y, cos, sin, pairs):
    """y [B, N, H, 64] with its first 2 h dims turned by the angles of cos, sin [.., N, 1, h]."""
    h = cos.shape[-1]
    r = y[..., : 2 * h]
    a, b = (r[..., :h], r[..., h:]) if pairs == "halves" else (r[..., 0::2], r[..., 1::2])
    c, d = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([c, d], -1) if pairs == "halves" else torch.stack([c, d], -1).flatten(-2)
    return torch.cat([turned, y[..., 2 * h:]], -1)


def _angles(s):
    """cos and sin of every token, [.., N, 1, h]; a token at a negative place is not turned."""
    pos = s["pos"].long()
    off = (pos < 0)[..., None]
    cos, sin = s["cos"][pos.clamp(min=0)], s["sin"][pos.clamp(min=0)]
    return torch.where(off, torch.ones_like(cos), cos)[..., None, :], torch.where(off, torch.zeros_like(sin), sin)[..., None, :]


def _heads(s):
    c = s["case"]
    x = s["x"].view(c["B"], c["N"], c["Hq"] + 2 * c["Hk"], HEAD)
    return x.split([c["Hq"], c["Hk"], c["Hk"]], 2)


def _plain_norm_fwd(s):
    cos, sin = _angles(s)
    xq, xk, xv = _heads(s)
    out = []
    for x, w in ((xq, s["wq"]), (xk, s["wk"])):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_rotate(y, cos, sin, s["case"]["pairs"]).to(s["x"].dtype).transpose(1, 2).contiguous())
    return out[0], out[1], xv.transpose(1, 2).contiguous()


def _plain_norm_bwd(s):
    cos, sin = _angles(s)
    xq, xk, _ = _heads(s)
    dx, dw = [], []
    for x, w, dz in ((xq, s["wq"], s["dq"]), (xk, s["wk"], s["dk"])):
        x, w = x.float(), w.float()
        dy = _rotate(dz.transpose(1, 2).float(), cos, -sin, s["case"]["pairs"])
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r
        dw.append((dy * n).sum((0, 1, 2), dtype=torch.float64).to(s["wq"].dtype))
        g = dy * w
        dx.append((r * (g - n * (g * n).mean(-1, keepdim=True))).to(s["x"].dtype))
    dx.append(s["dv"].transpose(1, 2))
    return torch.cat(dx, 2).flatten(2), dw[0], dw[1]


def _weights(s):
    """Softmax weights [B, Hq, Nq, Nk] and the log of their sums, in 32 bits."""
    q, k = s["q"].float(), s["k"].float()
    B, Hq, Nq, _ = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    x = (q * s["scale"]).reshape(B, Hkv, Hq // Hkv * Nq, HEAD) @ k.transpose(-1, -2)
    x = x.view(B, Hq, Nq, Nk)
    out = None
    if s["len"] is not None:
        out = torch.arange(Nk, device=q.device)[None] >= s["len"][:, None]
    elif s["mask"] is not None:
        out = ~s["mask"]
    if out is not None:
        x = x.masked_fill_(out[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)
    return x.div_(torch.where(total == 0, torch.ones_like(total), total)), lse


def _plain_cross_fwd(s):
    p, lse = _weights(s)
    B, Hq, Nq, Nk = p.shape
    v = s["v"].float()
    o = p.view(B, v.shape[1], -1, Nk) @ v
    # in the queries' layout, [B, N, H, 64] underneath
    return o.view(B, Hq, Nq, HEAD).to(s["q"].dtype).transpose(1, 2).contiguous().transpose(1, 2), lse


def _plain_cross_bwd(s):
    p, _ = _weights(s)
    B, Hq, Nq, Nk = p.shape
    t, Hkv = s["q"].dtype, s["k"].shape[1]
    k, v = s["k"].float(), s["v"].float()
    do = s["do"].float().reshape(B, Hkv, -1, HEAD)
    q = s["q"].float().reshape(B, Hkv, -1, HEAD)
    p = p.view(B, Hkv, -1, Nk)
    dv = p.transpose(-1, -2) @ do
    ds = do @ v.transpose(-1, -2)
    ds = ds.sub_((p * ds).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k) * s["scale"]
    dk = (ds.transpose(-1, -2) @ q) * s["scale"]
    return dq.view(B, Hq, Nq, HEAD).to(t), dk.to(t), dv.to(t)


# --------------------------------------------------------------------- calls

def _own(s):
    from sparse_head_self_gb300 import api
    op = s["case"]["op"]
    if op.startswith("norm"):
        c = s["case"]
        how = {"eps": EPS, "rotary": (s["cos"], s["sin"]), "positions": s["pos"], "interleaved": c["pairs"] == "neighbours"}
        heads = (c["Hq"], c["Hk"], c["Hk"])
        if op == "norm_fwd":
            return api.qk_norm_fwd(s["x"], heads, s["wq"], s["wk"], **how)
        return api.qk_norm_bwd(s["x"], heads, s["wq"], s["wk"], s["dq"], s["dk"], s["dv"], **how)
    how = {"kv_len": s["len"], "key_mask": s["mask"]}
    if op == "cross_fwd":
        return api.cross_fwd(s["q"], s["k"], s["v"], s["scale"], **how)
    return api.cross_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["scale"], **how)


def run(state):
    if own:
        return _own(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "cross_fwd": _plain_cross_fwd,
            "cross_bwd": _plain_cross_bwd}[state["case"]["op"]](state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, Hq = case["B"], case["Hq"]
    if case["op"].startswith("norm"):
        N, Hk = case["N"], case["Hk"]
        table = min(N, 16385) * case["rot"] * 4
        rows = B * N * HEAD * e
        if case["op"] == "norm_fwd":
            return {"bytes": rows * 2 * (Hq + 2 * Hk) + table, "flops": 9 * B * N * HEAD * (Hq + Hk)}
        # the values' part of x is not needed
        return {"bytes": rows * (3 * (Hq + Hk) + 2 * Hk) + table, "flops": 16 * B * N * HEAD * (Hq + Hk)}
    Hkv, Nq, Nk = case["Hkv"], case["Nq"], case["Nk"]
    keys = sum(_lengths(case)) if case["mask"] == "len" else B * (_kept(case) if case["mask"] == "mask" else Nk)
    pairs = keys * Hq * Nq
    qrows, krows = B * Hq * Nq, keys * Hkv
    if case["op"] == "cross_fwd":
        return {"bytes": e * HEAD * 2 * (qrows + krows) + 4 * qrows, "flops": 4 * HEAD * pairs}
    return {"bytes": e * HEAD * (4 * qrows + 2 * krows + 2 * B * Nk * Hkv) + 4 * qrows, "flops": 10 * HEAD * pairs}


# ------------------------------------------------- the definition in 64 bits

def _turn64(s, x, w, back=None):
    """Definition of the norm and the rotation of heads x [B, N, H, 64]; with `back`, the
    gradients of <back, result> with respect to x and w."""
    c = s["case"]
    x = x.double()
    w = w.double()
    if back is not None:
        x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
    y = x / (x.pow(2).sum(-1, keepdim=True) / HEAD + EPS).sqrt() * w
    half = c["rot"] // 2
    pos = s["pos"].long().expand(c["B"], c["N"])
    cos = torch.ones(c["B"], c["N"], 1, half, device=x.device, dtype=torch.float64)
    sin = torch.zeros_like(cos)
    at = pos >= 0
    cos[at] = s["cos"].double()[pos[at]][:, None]
    sin[at] = s["sin"].double()[pos[at]][:, None]
    i = torch.arange(half, device=x.device)
    first, second = (i, i + half) if c["pairs"] == "halves" else (2 * i, 2 * i + 1)
    z = y.clone()
    z[..., first] = cos * y[..., first] - sin * y[..., second]
    z[..., second] = sin * y[..., first] + cos * y[..., second]
    if back is None:
        return z
    return torch.autograd.grad(z, (x, w), back)


def _exact_norm(s):
    c = s["case"]
    Hq, Hk = c["Hq"], c["Hk"]
    x = s["x"].view(c["B"], c["N"], -1, HEAD)
    if c["op"] == "norm_fwd":
        return (_turn64(s, x[:, :, :Hq], s["wq"]).transpose(1, 2), _turn64(s, x[:, :, Hq:Hq + Hk], s["wk"]).transpose(1, 2),
                x[:, :, Hq + Hk:].double().transpose(1, 2))
    dxq, dwq = _turn64(s, x[:, :, :Hq], s["wq"], s["dq"].double().transpose(1, 2))
    dxk, dwk = _turn64(s, x[:, :, Hq:Hq + Hk], s["wk"], s["dk"].double().transpose(1, 2))
    return torch.cat([dxq, dxk, s["dv"].double().transpose(1, 2)], 2).reshape(c["B"], c["N"], -1), dwq, dwk


def _exact_cross(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, Hq, Nq, _ = q.shape
    Hkv, Nk = k.shape[1:3]
    o = torch.zeros(B, Hq, Nq, HEAD, device=q.device, dtype=torch.float64)
    lse = torch.full((B, Hq, Nq), -math.inf, device=q.device, dtype=torch.float64)
    dq = torch.zeros_like(o)
    dk = torch.zeros(B, Hkv, Nk, HEAD, device=q.device, dtype=torch.float64)
    dv = torch.zeros_like(dk)
    for b in range(B):
        keep = torch.ones(Nk, dtype=torch.bool, device=q.device)
        if s["len"] is not None:
            keep = torch.arange(Nk, device=q.device) < s["len"][b]
        if s["mask"] is not None:
            keep = keep & s["mask"][b]
        at = keep.nonzero().squeeze(1)
        if not len(at):
            continue
        for h in range(Hq):
            u = h // (Hq // Hkv)
            qq, kk, vv = q[b, h].double(), k[b, u, at].double(), v[b, u, at].double()
            x = s["scale"] * (qq @ kk.T)
            lse[b, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[b, h, :, None])
            o[b, h] = p @ vv
            if s["case"]["op"] == "cross_bwd":
                g = s["do"][b, h].double()
                dp = g @ vv.T
                ds = p * (dp - (g * o[b, h]).sum(-1, keepdim=True))
                dq[b, h] = s["scale"] * (ds @ kk)
                dk[b, u, at] += s["scale"] * (ds.T @ qq)
                dv[b, u, at] += p.T @ g
    return (o, lse) if s["case"]["op"] == "cross_fwd" else (dq, dk, dv)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"].startswith("norm") else _exact_cross(s)
