"""The paged 8-bit cache from its definition: pages simulated in 64 bits, value by
value, and the attention to what they hold with a bound on how far the kernel's may be
from it.

Storing and loading have no tolerance: scales, bytes and loaded values are
equal.  The attention's bounds count, with u = 2^-24 and h = eps / 2 of the I/O type:
  score     64 products summed within the instructions, whose additions are cut off (a whole step, 2 u,
            each), and scaled (3 u): 134 u of the terms' sizes; in 32 bits 4 u more for queries of 22 bits;
            and 2^-33 of the row's largest query value times the keys' sizes (a half's smallest step)
  weight    relative: the exponent's error, 2^-22 of the exponential, and 2^-11 (bf16) or 2^-22 (fp32) of
            its rounding; absolute: 2^-32 of the row's largest (a half's smallest step)
  sums      2 n u of the sum of sizes over n keys
  result    h of its own value
"""
import math

import torch

U = 2.0 ** -24
PAGE = 64

# The values of the bytes 0 to 126 (127 is NaN, the upper half the same with a sign).
VALUES = torch.tensor([math.ldexp(i % 8 + (8 if i >= 8 else 0), max(i // 8, 1) - 10) for i in range(127)], dtype=torch.float64)


def nearest(x):
    """The byte of the representable value nearest to each x (64 bits, CPU)."""
    a = x.abs().clamp(max=448.0).nan_to_num(0.0).contiguous()
    hi = torch.searchsorted(VALUES, a).clamp(1, 126)
    up, down = VALUES[hi] - a, a - VALUES[hi - 1]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    code = torch.where(x.isnan(), torch.full_like(code, 127), code)
    return (code + 128 * torch.signbit(x).long()).to(torch.uint8)


def decode(byte):
    code = byte.long() % 128
    v = torch.where(code == 127, torch.full((), math.nan, dtype=torch.float64), VALUES[code.clamp(max=126)])
    return torch.where(byte >= 128, -v, v)


def scale_of(values):
    """The smallest power of two whose 448th multiple reaches the largest finite value."""
    top = max([abs(x) for x in values.flatten().tolist() if math.isfinite(x)], default=0.0)
    if top == 0.0:
        return 2.0 ** -100
    e = math.frexp(top)[1] - 10          # 448 2^e < top / 2 at the start
    while 448.0 * 2.0 ** e < top:
        e += 1
    return 2.0 ** max(e, -100)


def read_scale(s):
    """What a scale is read as: a power of two within the bounds as it is, another number as the
    power of two at or below its size, within the bounds, infinities and NaN as the largest."""
    if math.isnan(s) or math.isinf(s):
        return 2.0 ** 120
    return 2.0 ** max(-100, min(120, math.frexp(s)[1] - 1)) if s else 2.0 ** -100


class Pages:
    """What a cache's memory holds, on the CPU."""

    def __init__(self, data, scales):
        self.data, self.scales = data.cpu().clone(), scales.cpu().clone()

    def store(self, table, K, V, start=None, count=None):
        table = table.tolist()
        B, Hkv, N, _ = K.shape
        for b in range(B):
            s, n = (0 if start is None else int(start[b])), (N if count is None else max(0, min(N, int(count[b]))))
            for slot in range(s // PAGE, (s + n - 1) // PAGE + 1 if n else s // PAGE):
                if not 0 <= slot < len(table[b]) or not 0 <= table[b][slot] < len(self.data):
                    continue
                page, lo, hi = table[b][slot], max(s, slot * PAGE), min(s + n, (slot + 1) * PAGE)
                for h in range(Hkv):
                    for kind, src in enumerate((K, V)):
                        self._piece(page, h, kind, src[b, h, lo - s:hi - s].double().cpu(), lo - slot * PAGE)

    def _piece(self, page, h, kind, new, at):
        old = self.data[page, h, kind].view(PAGE, 64)
        old = old if kind == 0 else old.T           # [token, dim], a view
        need, had = scale_of(new), read_scale(float(self.scales[page, h, kind]))
        step = need if at == 0 else max(need, had)
        if at and step > had:
            old[:at] = nearest(decode(old[:at]) * (had / step))
        old[at:at + len(new)] = nearest(new / step)
        if at == 0 or step > had:
            self.scales[page, h, kind] = step

    def load(self, table, N, start=None, count=None):
        """K, V [B, Hkv, N, 64] in 64 bits."""
        table = table.tolist()
        B, Hkv = len(table), self.data.shape[1]
        out = torch.zeros(2, B, Hkv, N, 64, dtype=torch.float64)
        for b in range(B):
            s, n = (0 if start is None else int(start[b])), (N if count is None else max(0, min(N, int(count[b]))))
            for i in range(n):
                slot, t = (s + i) // PAGE, (s + i) % PAGE
                if 0 <= slot < len(table[b]) and 0 <= table[b][slot] < len(self.data):
                    piece = self.data[table[b][slot]].view(Hkv, 2, PAGE, 64)
                    f = torch.tensor([[read_scale(x) for x in row] for row in self.scales[table[b][slot]].tolist()]).double()
                    out[0, b, :, i] = decode(piece[:, 0, t]) * f[:, :1]
                    out[1, b, :, i] = decode(piece[:, 1, :, t]) * f[:, 1:]
        return out[0], out[1]


def attend(q, k, v, scale, seen):
    """{name: (value, bound)} of O and LSE: queries q [B, Hq, N, 64] on keys and values k, v
    [B, Hkv, T, 64] in 64 bits, where seen [B, N, T]."""
    dt = q.dtype
    h = torch.finfo(dt).eps / 2
    hw = 2.0 ** -11 if dt == torch.bfloat16 else 2.0 ** -22
    B, Hq, N, _ = q.shape
    G, T = Hq // k.shape[1], k.shape[2]
    some, used = seen.any(2)[:, None], seen.any(1)[:, None, :, None]
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    Q = torch.where(some[..., None], q.double(), zero)
    K = torch.where(used, k, zero).repeat_interleave(G, 1)
    V = torch.where(used, v, zero).repeat_interleave(G, 1)
    s = (scale * (Q @ K.transpose(-1, -2))).masked_fill_(~seen[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    base = torch.where(some.expand_as(lse), lse, zero)
    p = torch.exp(s - base[..., None])
    O = p @ V
    mag = abs(scale) * (Q.abs() @ K.abs().transpose(-1, -2)).amax(-1)
    floor = abs(scale) * 2.0 ** -33 * Q.abs().amax(-1) * K.abs().sum(-1).amax(-1)[..., None]
    ew = U * ((138 + 4) * mag + 4 * base.abs() + 8) + floor
    es = ew + U * (2 * T + 8)
    A = p @ V.abs()
    least = 2.0 ** -32 * p.amax(-1, keepdim=True) * (seen[:, None].double() @ V.abs())
    out = {"O": (O, 1.05 * (h * O.abs() + (hw + 2 * es)[..., None] * A + least) + 1e-30),
           "LSE": (torch.where(some.expand_as(lse), lse, torch.full_like(lse, -math.inf)),
                   1.05 * (es + U * (2 * base.abs() + 16)))}
    return out
