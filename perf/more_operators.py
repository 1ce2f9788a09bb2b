"""Attention over a sliding window with sinks, its gradient, and a paged cache of
keys and values in 8 bits with the attention that reads it: their plain forms,
their calls, and the cases they are measured on.

A case is a dict of plain values:

  op       "win_fwd", "win_bwd": causal attention of Nq queries, the last of Nk
           tokens, to the `window` tokens that end with their own and to the
           first `sinks` tokens, and its gradient
           "store": N tokens' keys and values into the pages of a cache; what
           the pages then hold comes back as the values it stands for
           "cache_fwd": attention of the Nq newest tokens to such a cache
  dtype    "bf16" or "f32", the type of every tensor but the statistics and
           the cache
  window   0: every token up to the query's own
  ragged   the sequences have lengths of their own, where there are at least
           four one of them none
"""
import math

import torch

own = False

HEAD = 64
PAGE = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = 448.0          # of the 8-bit type


def _win(name, op, dtype, B, Hq, Hkv, Nq, Nk, window, sinks, ragged):
    c = {"op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "window": window, "sinks": sinks,
         "ragged": ragged}
    return {"name": name, **c} if name else c


def _store(name, dtype, B, Hkv, N, past):
    c = {"op": "store", "dtype": dtype, "B": B, "Hkv": Hkv, "N": N, "past": past}
    return {"name": name, **c} if name else c


def _cache(name, dtype, B, Hq, Hkv, Nq, T, window, sinks):
    c = {"op": "cache_fwd", "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "T": T, "window": window, "sinks": sinks}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the next token of sixteen sequences on their 16-bit keys, four query heads to a key head
        _win("win_fwd_token", "win_fwd", "bf16", 16, 16, 4, 1, 16385, 1024, 4, True),
        # a batch of short sequences, padded to the longest
        _win("win_fwd_short", "win_fwd", "bf16", 64, 12, 12, 197, 197, 64, 1, True),
        # training on the tokens of eight clips
        _win("win_fwd_clip", "win_fwd", "bf16", 8, 12, 4, 1569, 1569, 512, 4, True),
        # a part of two long prompts, whose earlier tokens are there
        _win("win_fwd_chunk", "win_fwd", "bf16", 2, 16, 4, 1569, 16385, 4096, 4, True),
        # training on one long sequence
        _win("win_fwd_long", "win_fwd", "bf16", 1, 16, 4, 16385, 16385, 1024, 4, False),
        # the gradients of the two training cases, ...
        _win("win_bwd_clip", "win_bwd", "bf16", 8, 12, 4, 1569, 1569, 512, 4, True),
        _win("win_bwd_long", "win_bwd", "bf16", 1, 16, 4, 16385, 16385, 1024, 4, False),
        # ... and of a small model in 32 bits
        _win("win_bwd_f32", "win_bwd", "f32", 4, 12, 12, 197, 197, 65, 1, True),
        # the prompts of eight sequences go into an empty cache
        _store("store_prompt", "bf16", 8, 4, 1569, 0),
        # one new token of each of 64 sequences
        _store("store_token", "bf16", 64, 4, 1, 1569),
        # one token of sixteen sequences on everything that they hold
        _cache("cache_token_long", "bf16", 16, 16, 4, 1, 16385, 0, 0),
        # four tokens each of 64 sequences (a guess that is verified) on the window and the sinks
        _cache("cache_few_window", "bf16", 64, 16, 4, 4, 16385, 1024, 4),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["win_fwd", "win_fwd", "win_bwd", "win_bwd", "store", "cache_fwd", "cache_fwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 3, 4, 12, 16])
    Hq = Hkv * rng.choice([1, 1, 2, 3, 4])
    window = 0 if rng.random() < 0.2 else _spread(rng, 16, 4096)
    sinks = rng.choice([0, 1, 4, 4, 16, 100])
    if kind == "store":
        while True:
            B, N = _spread(rng, 1, 64), 1 if rng.random() < 0.3 else _spread(rng, 2, 4096)
            if B * N * Hkv <= 8 * 1569 * 4:
                return _store(None, dtype, B, Hkv, N, 0 if rng.random() < 0.3 else _spread(rng, 1, 4096))
    if kind == "cache_fwd":
        while True:
            B, T = _spread(rng, 1, 64), _spread(rng, 16, 16385)
            Nq = 1 if rng.random() < 0.6 else rng.randint(2, 16)
            if B * T * Hkv <= 16 * 16385 * 4 and Hq // Hkv * Nq <= 64 and Nq <= T:
                return _cache(None, dtype, B, Hq, Hkv, Nq, T, window, sinks)
    while True:
        B, Nk = _spread(rng, 1, 64), _spread(rng, 3, 16385)
        Nq = Nk if rng.random() < 0.5 else _spread(rng, 1, Nk)
        if kind == "win_fwd" and rng.random() < 0.25:
            Nq = 1
        c = _win(None, kind, dtype, B, Hq, Hkv, Nq, Nk, window, sinks, rng.random() < 0.5)
        # of the largest listed ones; the 32-bit path is for smaller models
        dense, pairs = (16 * 16385 * 16385, 16 * 16385 * 1028) if dtype == "bf16" else (8 * 12 * 1569 * 1569, 8 * 12 * 1569 * 516)
        if B * Hq * Nq * Nk <= dense and Hq * _pairs(c) <= pairs and B * Hkv * Nk <= 16 * 4 * 16385:
            return c


# ------------------------------------------------------------------- inputs

def _lengths(case):
    """Lengths of the sequences, the same for every seed but for their order."""
    B, most = case["B"], case["Nk"] if case["op"].startswith("win") else case["T"]
    if case["op"].startswith("win") and not case["ragged"]:
        return [most] * B
    lens = [max(1, round(most * (1.0 - 0.5 * i / max(1, B - 1)))) for i in range(B)]
    if B >= 4 and case["op"].startswith("win"):
        lens[-1] = 0   # a sequence that is already finished
    return lens


def _starts(case, lens):
    """Positions of the sequences' first queries."""
    return [0 if case.get("Nq") == case.get("Nk") else n - case["Nq"] for n in lens]


def _e4m3(x):
    """The 8-bit values nearest to x, as bytes."""
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = TYPES[case["dtype"]]
    B, Hkv = case["B"], case["Hkv"]

    def randn(*shape, dtype=t):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    def int32(values):
        return torch.tensor(values, device=dev, dtype=torch.int32)

    s = {"case": case}
    order = torch.randperm(B, generator=g, device=dev)
    if case["op"].startswith("win"):
        Hq, Nq, Nk = case["Hq"], case["Nq"], case["Nk"]
        # as the projections leave them: queries [B, N, H, 64], keys and values side by side
        s["q"] = randn(B, Nq, Hq, HEAD).transpose(1, 2)
        kv = randn(B, Nk, 2, Hkv, HEAD)
        s["k"], s["v"] = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
        s["scale"] = HEAD ** -0.5
        lens = _lengths(case)
        s["start"] = int32(_starts(case, lens))[order].contiguous() if case["ragged"] and Nq < Nk else None
        s["len"] = int32(lens)[order].contiguous() if case["ragged"] else None
        if case["op"] == "win_bwd":
            s["do"] = randn(B, Nq, Hq, HEAD).transpose(1, 2)
            s["o"], s["lse"] = _plain_win_fwd(s)
        return s
    # Keys' dims differ in size, as they do after training.
    size = torch.exp(0.5 * randn(2, Hkv, 1, HEAD, dtype=torch.float32))

    def states(N):
        """Keys and values [B, Hkv, N, 64] of N tokens, side by side."""
        kv = (torch.randn(B, N, 2, Hkv, HEAD, generator=g, device=dev) * size[:, :, 0]).to(t)
        return kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)

    if case["op"] == "store":
        N, past = case["N"], case["past"]
        starts = [max(0, past - (37 * i) % (past + 1)) for i in range(B)]
        held = past + N
    else:
        held = case["T"]
        starts = [n - case["Nq"] for n in _lengths(case)]
    s["start"] = int32(starts)[order].contiguous()
    # Pages handed out over time, so that a sequence's lie anywhere; the last one is nobody's.
    M = (held + PAGE - 1) // PAGE
    s["table"] = torch.randperm(B * M, generator=g, device=dev).to(torch.int32).view(B, M)
    # what the sequences hold already
    past = torch.randn(B * M + 1, Hkv, 2, PAGE, HEAD, generator=g, device=dev) * size.transpose(0, 1)
    s["scales"] = _step(past.abs().amax((3, 4)))
    past[:, :, 1] = past[:, :, 1].transpose(2, 3).clone()
    s["data"] = _e4m3(past / s["scales"][..., None, None]).flatten(3).contiguous()
    if case["op"] == "store":
        s["k"], s["v"] = states(case["N"])
        s["from"] = s["start"] // PAGE * PAGE       # of the pages that the tokens go to
        s["count"] = s["start"] - s["from"] + case["N"]
        return s
    s["q"] = randn(B, case["Nq"], case["Hq"], HEAD).transpose(1, 2)
    s["scale"] = HEAD ** -0.5
    return s


# --------------------------------------------------------------- plain forms

def _visible(p, k, length, window, sinks):
    """Whether the queries at positions p [.., Nq, 1] see the keys k [Nk]."""
    seen = (k <= p) & (k < length) & (p < length)
    return seen if window == 0 else seen & ((k > p - window) | (k < sinks))


def _weights(x, seen):
    """Softmax of x [B, H, N, K] over the keys that are seen [B, 1, N, K], and the logs of the sums; x is overwritten."""
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)
    return x.div_(torch.where(total == 0, torch.ones_like(total), total)), lse


def _win_weights(s):
    c = s["case"]
    q, k = s["q"].float(), s["k"].float()
    B, Hq, Nq, _ = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    x = (q * s["scale"]).reshape(B, Hkv, Hq // Hkv * Nq, HEAD) @ k.transpose(-1, -2)
    start = torch.full((B,), Nk - Nq, device=q.device) if s["start"] is None else s["start"].long()
    length = torch.full((B,), Nk, device=q.device) if s["len"] is None else s["len"].long()
    p = start[:, None, None, None] + torch.arange(Nq, device=q.device)[:, None]
    seen = _visible(p, torch.arange(Nk, device=q.device), length[:, None, None, None], c["window"], c["sinks"])
    return _weights(x.view(B, Hq, Nq, Nk), seen)


def _values(p, v, t):
    """p [B, Hq, N, K] times v [B, Hkv, K, 64], in the queries' layout, [B, N, H, 64] underneath."""
    B, Hq, Nq, Nk = p.shape
    o = p.view(B, v.shape[1], -1, Nk) @ v
    return o.view(B, Hq, Nq, HEAD).to(t).transpose(1, 2).contiguous().transpose(1, 2)


def _plain_win_fwd(s):
    p, lse = _win_weights(s)
    return _values(p, s["v"].float(), s["q"].dtype), lse


def _plain_win_bwd(s):
    p, _ = _win_weights(s)
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


def _step(top):
    """The smallest power of two whose multiples by LARGEST reach `top` (2^-100 at least)."""
    m, e = torch.frexp(top)          # top = m 2^e, m in [0.5, 1)
    e = torch.where(m > LARGEST / 512, e - 8, e - 9)
    return ((e.clamp(min=-100) + 127) << 23).to(torch.int32).view(torch.float32)     # 2^e to the last bit


def _pages(data, scales):
    """The values [.., 2, 64 tokens, 64] of pages [.., 2, 4096]: keys lie token by token, values dim by dim."""
    x = data.view(torch.float8_e4m3fn).float().unflatten(-1, (PAGE, HEAD)) * scales[..., None, None]
    return torch.stack([x[..., 0, :, :], x[..., 1, :, :].transpose(-1, -2)], -3)


def _plain_load(s, first, N, count):
    """Keys and values [B, N, Hkv, 64] in 32 bits of the tokens from `first` on; zeros from `count` on."""
    n = torch.arange(N, device=first.device)
    pos = first.long()[:, None] + n
    page = s["table"].gather(1, (pos // PAGE).clamp(max=s["table"].shape[1] - 1)).long()
    tok = pos % PAGE
    d = s["data"].view(torch.float8_e4m3fn).unflatten(-1, (PAGE, HEAD))
    there = (n < count[:, None])[..., None, None]
    out = []
    for x, i in ((d[page, :, 0, tok], 0), (d[page, :, 1, :, tok], 1)):
        out.append(torch.where(there, x.float() * s["scales"][page, :, i][..., None], torch.zeros((), device=x.device)))
    return out


def _plain_store(s):
    B, Hkv, N, _ = s["k"].shape
    t, dev = s["k"].dtype, s["k"].device
    M, spare = s["table"].shape[1], s["data"].shape[0] - 1
    start = s["start"].long()[:, None]
    slot = start // PAGE + torch.arange((N + 126) // PAGE, device=dev)            # [B, S]
    used = slot * PAGE < start + N
    page = torch.where(used, s["table"].gather(1, slot.clamp(max=M - 1)).long(), torch.full_like(slot, spare))
    data, scales = s["data"][page], s["scales"][page]                             # [B, S, Hkv, 2, ..]
    n = (slot * PAGE)[..., None] + torch.arange(PAGE, device=dev) - start[..., None]    # [B, S, 64]
    kv = torch.stack([s["k"], s["v"]], 2).float().permute(0, 3, 1, 2, 4)          # [B, N, Hkv, 2, 64]
    new = kv[torch.arange(B, device=dev)[:, None, None], n.clamp(0, N - 1)].permute(0, 1, 3, 4, 2, 5)
    is_new = ((n >= 0) & (n < N))[:, :, None, None, :, None]
    is_old = (n < 0)[:, :, None, None, :, None]
    size = torch.where(is_new & new.isfinite(), new.abs(), torch.zeros((), device=dev)).amax((4, 5))
    step = _step(size)
    step = torch.where(is_old.any(4)[..., 0], torch.maximum(step, scales), step)
    step = torch.where(used[..., None, None], step, scales)
    x = torch.where(is_new, new, _pages(data, scales))
    x = _e4m3((x / step[..., None, None]).clamp(-LARGEST, LARGEST))
    x = torch.stack([x[..., 0, :, :], x[..., 1, :, :].transpose(-1, -2)], -3)
    behind = (n >= N)[:, :, None, None, None, :]
    behind = torch.cat([behind.transpose(-1, -2).expand(-1, -1, -1, -1, -1, HEAD), behind.expand(-1, -1, -1, -1, HEAD, -1)], 3)
    x = torch.where(behind, data.unflatten(-1, (PAGE, HEAD)), x)
    s["data"][page] = x.flatten(-2)
    s["scales"][page] = step
    return [x.to(t).transpose(1, 2).contiguous() for x in _plain_load(s, s["from"], N + PAGE - 1, s["count"])]


def _plain_cache_fwd(s):
    c = s["case"]
    B, Hq, Nq, _ = s["q"].shape
    T = s["table"].shape[1] * PAGE
    zero = torch.zeros(B, dtype=torch.int64, device=s["q"].device)
    k, v = (x.transpose(1, 2) for x in _plain_load(s, zero, T, s["start"].long() + Nq))
    x = (s["q"].float() * s["scale"]).reshape(B, c["Hkv"], -1, HEAD) @ k.transpose(-1, -2)
    p = s["start"].long()[:, None, None, None] + torch.arange(Nq, device=x.device)[:, None]
    p, lse = _weights(x.view(B, Hq, Nq, T), _visible(p, torch.arange(T, device=x.device), T, c["window"], c["sinks"]))
    return _values(p, v, s["q"].dtype), lse


# --------------------------------------------------------------------- calls

def _own(s):
    from sparse_head_self_gb300 import api
    c = s["case"]
    if c["op"] == "store":
        cache = api.Cache(s["data"], s["scales"])
        api.cache_store(cache, s["table"], s["k"], s["v"], s["start"])
        return api.cache_load(cache, s["table"], c["N"] + PAGE - 1, s["from"], s["count"], dtype=s["k"].dtype)
    band = {"window": c["window"] or None, "sinks": c["sinks"]}
    if c["op"] == "cache_fwd":
        return api.cache_fwd(s["q"], api.Cache(s["data"], s["scales"]), s["table"], s["start"], s["scale"], **band)
    band |= {"q_start": s["start"], "kv_len": s["len"]}
    if c["op"] == "win_fwd":
        return api.window_fwd(s["q"], s["k"], s["v"], s["scale"], **band)
    return api.window_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["scale"], **band)


def run(state):
    if own:
        return _own(state)
    return {"win_fwd": _plain_win_fwd, "win_bwd": _plain_win_bwd, "store": _plain_store,
            "cache_fwd": _plain_cache_fwd}[state["case"]["op"]](state)


def _ramp(n, most):
    """The sum of min(i, most) over i = 1..n."""
    m = min(n, most)
    return m * (m + 1) // 2 + max(0, n - most) * most


def _seen(case, start, length):
    """(pairs of a query and a key that it sees, keys that any query sees, queries that see some) of one query head."""
    first, last = max(0, start), min(start + case["Nq"], length)       # positions of those queries: [first, last)
    if first >= last:
        return 0, 0, 0
    window, sinks = case["window"] or length + 1, case["sinks"] if case["window"] else 0
    pairs = _ramp(last, window) - _ramp(first, window)
    # sinks in front of the window: min(sinks, max(0, p + 1 - window))
    pairs += _ramp(max(0, last - window), sinks) - _ramp(max(0, first - window), sinks)
    oldest = max(0, first + 1 - window)
    return pairs, last - oldest + min(sinks, oldest), last - first


def _all_seen(case):
    lens = _lengths(case)
    return [sum(x) for x in zip(*(_seen(case, a, n) for a, n in zip(_starts(case, lens), lens)))]


def _pairs(case):
    return _all_seen(case)[0]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, Hkv = case["B"], case["Hkv"]
    if case["op"] == "store":
        # the tokens in, their bytes out, and out again as values
        rows = 2 * B * Hkv * case["N"] * HEAD
        return {"bytes": rows * (2 * e + 1), "flops": 2 * rows}
    Hq, Nq = case["Hq"], case["Nq"]
    pairs, keys, queries = _all_seen(case)
    if case["op"] == "cache_fwd":
        return {"bytes": 2 * keys * Hkv * HEAD + 2 * B * Hq * Nq * HEAD * e + 4 * B * Hq * Nq, "flops": 4 * HEAD * pairs * Hq}
    qrows, krows = B * Hq * Nq, keys * Hkv
    if case["op"] == "win_fwd":
        return {"bytes": e * HEAD * (queries * Hq + qrows + 2 * krows) + 4 * qrows, "flops": 4 * HEAD * pairs * Hq}
    return {"bytes": e * HEAD * (3 * queries * Hq + qrows + 2 * krows + 2 * B * case["Nk"] * Hkv) + 4 * queries * Hq,
            "flops": 10 * HEAD * pairs * Hq}


# ------------------------------------------------- the definition in 64 bits

def _attend(q, k, v, scale, start, length, window, sinks, do=None):
    """One query head on its keys and values, 256 queries at a time: (o, lse) or, with
    the gradient of o, (dq, dk, dv)."""
    N, dev = q.shape[0], q.device
    o, dq = torch.zeros(N, HEAD, device=dev, dtype=torch.float64), torch.zeros(N, HEAD, device=dev, dtype=torch.float64)
    lse = torch.full((N,), -math.inf, device=dev, dtype=torch.float64)
    dk, dv = torch.zeros(k.shape, device=dev, dtype=torch.float64), torch.zeros(k.shape, device=dev, dtype=torch.float64)
    for a in range(max(0, -start), min(N, length - start), 256):
        b = min(a + 256, N, length - start)
        lo = max(0, start + a - window + 1) if window else 0
        at = torch.cat([torch.arange(min(sinks, lo), device=dev), torch.arange(lo, start + b, device=dev)])
        p = torch.arange(start + a, start + b, device=dev)[:, None]
        hidden = at > p
        if window:
            hidden = hidden | ((p - at >= window) & (at >= sinks))
        x = scale * (q[a:b].double() @ k[at].double().T)
        x[hidden] = -math.inf
        lse[a:b] = torch.logsumexp(x, -1)
        w = torch.exp(x - lse[a:b, None])
        o[a:b] = w @ v[at].double()
        if do is None:
            continue
        y = do[a:b].double()
        dw = w * (y @ v[at].double().T - (y * o[a:b]).sum(-1, keepdim=True))
        dq[a:b] = scale * (dw @ k[at].double())
        dk[at] += scale * (dw.T @ q[a:b].double())
        dv[at] += w.T @ y
    return (o, lse) if do is None else (dq, dk, dv)


def _exact_win(s):
    c = s["case"]
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    starts = [c["Nk"] - c["Nq"]] * B if s["start"] is None else s["start"].tolist()
    lens = [c["Nk"]] * B if s["len"] is None else s["len"].tolist()
    heads = [[_attend(s["q"][b, h], s["k"][b, h * Hkv // Hq], s["v"][b, h * Hkv // Hq], s["scale"], starts[b], lens[b],
                      c["window"], c["sinks"], s["do"][b, h] if c["op"] == "win_bwd" else None) for h in range(Hq)]
             for b in range(B)]
    out = [torch.stack([torch.stack([x[i] for x in row]) for row in heads]) for i in range(len(heads[0][0]))]
    return out if c["op"] == "win_fwd" else [out[0], *(x.view(B, Hkv, Hq // Hkv, -1, HEAD).sum(2) for x in out[1:])]


def _codes(dev):
    """The values of the bytes 0 to 126: four bits of exponent, three behind the point."""
    return torch.tensor([math.ldexp(i % 8 + (8 if i >= 8 else 0), max(i // 8, 1) - 10) for i in range(127)], device=dev,
                        dtype=torch.float64)


def _nearest(x):
    """The representable values nearest to x, those with an even byte where two are as near."""
    codes = _codes(x.device)
    a = x.abs().clamp(max=LARGEST).contiguous()
    hi = torch.searchsorted(codes, a).clamp(1, 126)
    lo = hi - 1
    up, down = codes[hi] - a, a - codes[lo]
    i = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(codes[i], x)


def _held(s, page):
    """Keys and values [64, Hkv, 2, 64] that a page holds, and its scales."""
    x = s["data"][page].long()
    v = _codes(x.device)[(x % 128).clamp(max=126)] * torch.where(x < 128, 1.0, -1.0).double()
    v = v.view(-1, 2, 64, 64) * s["scales"][page].double()[..., None, None]
    return torch.stack([v[:, 0].permute(1, 0, 2), v[:, 1].permute(2, 0, 1)], 2), s["scales"][page].double()


def _exact_store(s):
    c = s["case"]
    B, Hkv, N = c["B"], c["Hkv"], c["N"]
    out = torch.zeros(2, B, Hkv, N + PAGE - 1, HEAD, device=s["data"].device, dtype=torch.float64)
    for b, start in enumerate(s["start"].tolist()):
        first = start // PAGE
        for slot in range(first, (start + N - 1) // PAGE + 1):
            old, step = _held(s, int(s["table"][b, slot]))
            lo, hi = max(start, slot * PAGE), min(start + N, (slot + 1) * PAGE)
            new = torch.stack([s["k"][b, :, lo - start:hi - start], s["v"][b, :, lo - start:hi - start]], 2).double()
            new = new.transpose(0, 1)                                   # [tokens, Hkv, 2, 64]
            x = torch.cat([old[:lo - slot * PAGE], new])
            need = torch.tensor([[math.ldexp(1.0, math.frexp(x)[1] - (math.frexp(x)[0] == 0.5)) for x in row]
                                 for row in (new.abs().amax((0, 3)) / LARGEST).tolist()], device=step.device, dtype=torch.float64)
            step = torch.maximum(step, need) if lo > slot * PAGE else need
            at = (slot - first) * PAGE
            out[:, b, :, at:at + len(x)] = (_nearest(x / step[..., None]) * step[..., None]).permute(2, 1, 0, 3)
    return [out[0], out[1]]


def _exact_cache(s):
    c = s["case"]
    B, Hq, Hkv, Nq = c["B"], c["Hq"], c["Hkv"], c["Nq"]
    o, lse = [], []
    for b, start in enumerate(s["start"].tolist()):
        n = (start + Nq + PAGE - 1) // PAGE
        kv = torch.stack([_held(s, p)[0] for p in s["table"][b, :n].tolist()]).flatten(0, 1)      # [tokens, Hkv, 2, 64]
        heads = [_attend(s["q"][b, h], kv[:, h * Hkv // Hq, 0], kv[:, h * Hkv // Hq, 1], s["scale"], start, start + Nq,
                         c["window"], c["sinks"]) for h in range(Hq)]
        o.append(torch.stack([x[0] for x in heads]))
        lse.append(torch.stack([x[1] for x in heads]))
    return torch.stack(o), torch.stack(lse)


def exact(case, seed):
    s = prepare(case, seed)
    return {"win_fwd": _exact_win, "win_bwd": _exact_win, "store": _exact_store, "cache_fwd": _exact_cache}[case["op"]](s)
