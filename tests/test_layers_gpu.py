"""The layers with the query/key norm, the position rotation and the cross
attention, alone and together as an encoder-decoder: outputs and every
gradient against the same layers in torch operations, in 64 bits (their 32-bit
run is the tolerance: a kernel's run may be a few times as far off)."""
import os
import subprocess
import sys

import pytest
import torch

import oracle
from sparse_head_self_gb300 import api
from sparse_head_self_gb300.block import CrossAttention, FibottentionSelfAttention

pytestmark = pytest.mark.gpu


def _turn(y, cos, sin, pos):
    """y [B, H, N, 64] turned by the tables at the positions [N] (halves paired)."""
    h = cos.shape[1]
    on = (pos >= 0)[:, None].to(y.dtype)
    c = cos.to(y.dtype)[pos.clamp(min=0)] * on + (1 - on)
    s = sin.to(y.dtype)[pos.clamp(min=0)] * on
    a, b = y[..., :h], y[..., h:2 * h]
    return torch.cat([a * c - b * s, a * s + b * c, y[..., 2 * h:]], -1)


def _norm(x, w, eps):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def _attend(q, k, v, scale, keep):
    G = q.shape[1] // k.shape[1]
    s = scale * q @ k.repeat_interleave(G, 1).transpose(-1, -2)
    p = torch.softmax(s.masked_fill(~keep, float("-inf")), -1).nan_to_num(0.0)
    return p @ v.repeat_interleave(G, 1)


def _self_ref(layer, x, masks):
    B, N, dim = x.shape
    q, k, v = layer.qkv(x).view(B, N, 3, layer.heads, 64).permute(2, 0, 3, 1, 4)
    q, k = _norm(q, layer.q_norm, layer.eps), _norm(k, layer.k_norm, layer.eps)
    if layer.rotary is not None:
        pos = torch.arange(N, device=x.device) if layer.positions is None else layer.positions.long()
        q, k = (_turn(t, *layer.rotary.tables(), pos) for t in (q, k))
    o = _attend(q, k, v, layer.scale, masks[None])
    return layer.proj(o.transpose(1, 2).reshape(B, N, dim))


def _cross_ref(layer, x, y, keep):
    B, Nq, dim = x.shape
    q = _norm(layer.q(x).view(B, Nq, layer.heads, 64).transpose(1, 2), layer.q_norm, layer.eps)
    k, v = layer.kv(y).view(B, y.shape[1], 2, layer.kv_heads, 64).permute(2, 0, 3, 1, 4)
    k = _norm(k, layer.k_norm, layer.eps)
    if layer.rotary is not None:
        q = _turn(q, *layer.rotary.tables(), torch.arange(Nq, device=x.device))
    if layer.state_rotary is not None:
        k = _turn(k, *layer.state_rotary.tables(), torch.arange(y.shape[1], device=x.device))
    o = _attend(q, k, v, layer.scale, keep[:, None, None])
    return layer.proj(o.transpose(1, 2).reshape(B, Nq, dim))


def _masks(H, N):
    w = oracle.windows(H, 5, N)
    heads = [oracle.Head.fibottention(*oracle.wythoff_row(i + 1), w[i], True, False) for i in range(H)]
    return torch.stack([torch.from_numpy(oracle.support_mask(N, h).astype(bool)) for h in heads]).cuda()


def _run(fn, inputs, layers, g):
    for layer in layers:
        layer.zero_grad()
    xs = [x.detach().clone().requires_grad_() for x in inputs]
    out = fn(*xs)
    out.backward(g.to(out.dtype))
    return [out.detach()] + [x.grad for x in xs] + [p.grad for layer in layers for p in layer.parameters()]


def _compare(own, plain, inputs, layers, g):
    """own and plain take (layers, *inputs)."""
    got = _run(lambda *x: own(layers, *x), inputs, layers, g)
    near = _run(lambda *x: plain(layers, *x), inputs, layers, g)
    for m in layers:      # in place: the layers' support handles are not copied
        m.double()
    want = _run(lambda *x: plain(layers, *x), [x.double() for x in inputs], layers, g)
    for i, (a, b, c) in enumerate(zip(got, near, want)):
        size = float(c.abs().max())
        off, ref = float((a.double() - c).abs().max()), float((b.double() - c).abs().max())
        assert off <= 8 * ref + 1e-5 * size, (i, off, ref, size)


@pytest.mark.parametrize("norm,rot,cls", [(True, True, True), (True, False, False), (False, True, False)])
def test_self_attention_layer(norm, rot, cls):
    torch.manual_seed(0)
    B, H, N = 2, 4, 65
    angles = api.rotary_angles_2d(8, 8) if cls else api.rotary_angles(N, 32)
    layer = FibottentionSelfAttention(H * 64, H, N, 5, N, norm=norm, rotary=angles if rot else None, class_token=cls).cuda()
    if norm:
        with torch.no_grad():
            layer.q_norm.add_(0.2 * torch.randn(64, device="cuda"))
            layer.k_norm.add_(0.2 * torch.randn(64, device="cuda"))
    m = _masks(H, N)
    x = torch.randn(B, N, H * 64, device="cuda")
    _compare(lambda ls, x: ls[0](x), lambda ls, x: _self_ref(ls[0], x, m), [x], [layer], torch.randn_like(x))


@pytest.mark.parametrize("kv_heads,norm,rot", [(4, True, True), (2, False, False), (1, True, False), (4, False, True)])
def test_cross_attention_layer(kv_heads, norm, rot):
    torch.manual_seed(1)
    B, H, Nq, Nk = 3, 4, 21, 65
    layer = CrossAttention(H * 64, H, 192, kv_heads, norm=norm, rotary=api.rotary_angles(40) if rot else None,
                           state_rotary=api.rotary_angles(Nk) if rot else None).cuda()
    x, y = torch.randn(B, Nq, H * 64, device="cuda"), torch.randn(B, Nk, 192, device="cuda")
    n = torch.tensor([65, 0, 17], dtype=torch.int32, device="cuda")
    keep = torch.arange(Nk, device="cuda")[None] < n[:, None]
    _compare(lambda ls, x, y: ls[0](x, y, kv_len=n), lambda ls, x, y: _cross_ref(ls[0], x, y, keep), [x, y], [layer],
             torch.randn_like(x))


def test_encoder_and_decoder_together():
    torch.manual_seed(2)
    B, H, N, Nq = 2, 3, 65, 33
    enc = FibottentionSelfAttention(H * 64, H, N, 5, N, norm=True, rotary=api.rotary_angles_2d(8, 8), class_token=True)
    dec = CrossAttention(H * 64, H, norm=True, rotary=api.rotary_angles(Nq), kv_heads=1)
    enc, dec = enc.cuda(), dec.cuda()
    m, keep = _masks(H, N), torch.rand(B, N, device="cuda") < 0.7
    image, text = torch.randn(B, N, H * 64, device="cuda"), torch.randn(B, Nq, H * 64, device="cuda")

    def own(ls, image, text):
        return ls[1](text, image + ls[0](image), key_mask=keep)

    def plain(ls, image, text):
        return _cross_ref(ls[1], text, image + _self_ref(ls[0], image, m), keep)

    _compare(own, plain, [image, text], [enc, dec], torch.randn_like(text))


def test_decoding_token_by_token():
    # the states' keys and values once, then one query a step: what the whole sequence gives
    torch.manual_seed(3)
    B, H, Nq, Nk = 2, 4, 6, 197
    layer = CrossAttention(H * 64, H, 128, kv_heads=2, norm=True, rotary=api.rotary_angles(Nq)).cuda()
    x, y = torch.randn(B, Nq, H * 64, device="cuda"), torch.randn(B, Nk, 128, device="cuda")
    n = torch.tensor([197, 60], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        whole = layer(x, y, kv_len=n)
        kv = layer.states(y)
        for i in range(Nq):
            at = torch.tensor([i], dtype=torch.int32, device="cuda")
            one = layer(x[:, i:i + 1], kv=kv, kv_len=n, positions=at)
            # two orders of the same 32-bit sums: 1024 roundings of 2^-24 at most between them
            assert float((one - whole[:, i:i + 1]).abs().max()) <= 1024 * 2.0 ** -24 * float(whole.abs().max())
    with pytest.raises(ValueError, match="either"):
        layer(x)


def test_layers_in_16_bits_keep_their_angles():
    torch.manual_seed(4)
    H, N = 3, 65
    enc = FibottentionSelfAttention(H * 64, H, N, 5, N, norm=True, rotary=api.rotary_angles(N)).cuda()
    dec = CrossAttention(H * 64, H, norm=True, rotary=api.rotary_angles(N)).cuda()
    x = torch.randn(2, N, H * 64, device="cuda")
    wide = dec(x, enc(x)).float()
    enc, dec = enc.to(torch.bfloat16), dec.to(torch.bfloat16)
    assert enc.rotary.cos.dtype == torch.float32 and enc.rotary.cos.is_cuda
    y = dec(x.bfloat16(), enc(x.bfloat16()))
    assert y.dtype == torch.bfloat16
    # ten roundings of activations and weights of 2^-8 each, most of them averaged out
    assert float((y.float() - wide).abs().mean()) <= 10 * 2.0 ** -8 * float(wide.abs().mean())


@pytest.mark.parametrize("norm", [True, False])
def test_places_make_no_difference_to_a_layer_that_does_not_rotate(norm):
    torch.manual_seed(6)
    layer = CrossAttention(128, 2, norm=norm).cuda()
    x, y = torch.randn(2, 5, 128, device="cuda"), torch.randn(2, 9, 128, device="cuda")
    at = torch.arange(5, device="cuda", dtype=torch.int32) + 100
    want = layer(x, y)
    assert torch.equal(layer(x, y, positions=at), want)
    kv = layer.states(y, positions=torch.arange(9, device="cuda", dtype=torch.int32))
    assert torch.equal(layer(x, kv=kv, positions=at), want)


@pytest.mark.parametrize("norm", [True, False])
def test_layers_under_autocast(norm):
    # autocast rounds inputs and weights where the layers in 16 bits hold them so: the same numbers
    torch.manual_seed(5)
    B, H, N, Nq = 2, 3, 65, 21
    rot = api.rotary_angles(N)

    def layers():
        return (FibottentionSelfAttention(H * 64, H, N, 5, N, norm=norm, rotary=rot),
                CrossAttention(H * 64, H, kv_heads=1, norm=norm, rotary=rot, state_rotary=rot))

    wide, short = [m.cuda() for m in layers()], [m.cuda() for m in layers()]
    for a, b in zip(wide, short):
        with torch.no_grad():
            for p in (a.q_norm, a.k_norm):
                if p is not None:
                    p.add_(0.2 * torch.randn(64, device="cuda"))
        b.load_state_dict(a.state_dict())
        b.bfloat16()
    x, y = torch.randn(B, N, H * 64, device="cuda"), torch.randn(B, Nq, H * 64, device="cuda")
    g = torch.randn(B, Nq, H * 64, device="cuda").bfloat16()
    with torch.autocast("cuda", dtype=torch.bfloat16):
        got = _run(lambda x, y: wide[1](y, wide[0](x)), [x, y], wide, g)
    want = _run(lambda x, y: short[1](y, short[0](x)), [x.bfloat16(), y.bfloat16()], short, g)
    assert len(got) == len(want) and got[0].dtype is torch.bfloat16
    for i, (a, b) in enumerate(zip(got, want)):
        assert a.dtype is (torch.bfloat16 if i == 0 else torch.float32), i
        assert torch.equal(a.float(), b.float()), i


FIRST_CALL = """
import sys, torch
from sparse_head_self_gb300 import api
what, dtype, Nq = sys.argv[1], getattr(torch, sys.argv[2]), int(sys.argv[3])
g = torch.Generator(device="cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
q, k, v, do = r(2, 4, Nq, 64), r(2, 2, 300, 64), r(2, 2, 300, 64), r(2, 4, Nq, 64)
x, w = r(2, Nq, 8 * 64), r(64)
tables = api.rotary_tables(api.rotary_angles(Nq, 64, device="cuda"))

def call():
    if what == "norm":
        out = api.qk_norm_fwd(x, (4, 2, 2), w, w, 1e-6, tables)
        return out + api.qk_norm_bwd(x, (4, 2, 2), w, w, *out, 1e-6, tables)
    o, lse = api.cross_fwd(q, k, v, 0.125)
    return (o, lse) + api.cross_bwd(q, k, v, o, lse, do, 0.125)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
assert all(torch.equal(a, b) for a, b in zip(got, call()))
assert all(bool(t.isfinite().all()) for t in got)
"""


@pytest.mark.parametrize("what,dtype,Nq", [("norm", "bfloat16", 40), ("cross", "bfloat16", 1), ("cross", "bfloat16", 150),
                                           ("cross", "float32", 1), ("cross", "float32", 150)])
def test_the_first_call_of_a_process_may_be_captured(what, dtype, Nq):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    child = subprocess.run([sys.executable, "-c", FIRST_CALL, what, dtype, str(Nq)], cwd=root, capture_output=True, text=True,
                           timeout=300)
    assert child.returncode == 0, child.stderr[-2000:]
