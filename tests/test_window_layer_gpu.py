"""The decoder's self-attention layer: outputs and every gradient against the same
layer in torch operations in 64 bits; decoding on the 8-bit cache, chunk by chunk and
token by token, against the definition on the values that the cache holds."""
import pytest
import torch

from test_layers_gpu import _attend, _compare, _cross_ref, _norm, _turn
from window_ref import seen_of
from sparse_head_self_gb300 import api
from sparse_head_self_gb300.block import CrossAttention, WindowSelfAttention

pytestmark = pytest.mark.gpu


def _layer(heads, kv_heads, norm, rot, window, sinks, seed=0):
    torch.manual_seed(seed)
    layer = WindowSelfAttention(heads * 64, heads, kv_heads, window, sinks, norm=norm,
                                rotary=api.rotary_angles(400, 32) if rot else None).cuda()
    if norm:
        with torch.no_grad():
            layer.q_norm.add_(0.2 * torch.randn(64, device="cuda"))
            layer.k_norm.add_(0.2 * torch.randn(64, device="cuda"))
    return layer


def _split_ref(layer, x, start=0):
    B, N, dim = x.shape
    H, G = layer.heads, layer.kv_heads
    q, k, v = layer.qkv(x).view(B, N, H + 2 * G, 64).transpose(1, 2).split((H, G, G), 1)
    q, k = _norm(q, layer.q_norm, layer.eps), _norm(k, layer.k_norm, layer.eps)
    if layer.rotary is not None:
        pos = torch.arange(start, start + N, device=x.device)
        q, k = (_turn(t, *layer.rotary.tables(), pos) for t in (q, k))
    return q, k, v


def _out(layer, o):
    return layer.proj(o.transpose(1, 2).flatten(2))


def _ref(layer, x, n=None):
    q, k, v = _split_ref(layer, x)
    seen = seen_of(x.shape[0], x.shape[1], x.shape[1], layer.window, layer.sinks, None, n)
    return _out(layer, _attend(q, k, v, layer.scale, seen[:, None]))


@pytest.mark.parametrize("kv_heads,norm,rot", [(4, True, True), (2, False, False), (1, True, False), (4, False, True)])
@pytest.mark.parametrize("band", [(None, 0), (20, 3)], ids=str)
def test_layer(kv_heads, norm, rot, band):
    layer = _layer(4, kv_heads, norm, rot, *band)
    x = torch.randn(3, 70, 256, device="cuda")
    n = torch.tensor([70, 33, 0], dtype=torch.int32, device="cuda")
    _compare(lambda ls, x: ls[0](x, n), lambda ls, x: _ref(ls[0], x, n), [x], [layer], torch.randn_like(x))


def test_decoder_of_both_attentions():
    # a decoder's block on an encoder's states: its own tokens, then the states
    own = _layer(4, 2, True, True, 30, 2, seed=3)
    other = CrossAttention(256, 4, kv_heads=2).cuda()
    x, y = torch.randn(2, 50, 256, device="cuda"), torch.randn(2, 65, 256, device="cuda")
    keep = torch.ones(2, 65, dtype=torch.bool, device="cuda")

    def run(ls, x, y):
        x = x + ls[0](x)
        return x + ls[1](x, y)

    def plain(ls, x, y):
        x = x + _ref(ls[0], x)
        return x + _cross_ref(ls[1], x, y, keep)

    _compare(run, plain, [x, y], [own, other], torch.randn_like(x))


@pytest.mark.parametrize("kv_heads,norm,rot", [(4, True, True), (2, False, False), (1, True, True)])
@pytest.mark.parametrize("band", [(None, 0), (90, 3)], ids=str)
def test_decoding_on_the_cache(kv_heads, norm, rot, band):
    layer = _layer(4, kv_heads, norm, rot, *band, seed=5)
    B, M = 2, 6
    cache = api.Cache.new(B * M, kv_heads)
    table = torch.randperm(B * M, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, M).cuda()
    x = torch.randn(B, 300, 256, device="cuda")
    at, chunks = 0, (130, 1, 1, 70, 5, 1, 40, 1)
    got = []
    for N in chunks:
        start = torch.full((B,), at, dtype=torch.int32, device="cuda")
        got.append((at, N, layer.step(x[:, at:at + N], cache, table, start), api.cache_load(cache, table, at + N, dtype=torch.float32)))
        at += N

    def reference(layer, x, at, N, kv):
        q = _split_ref(layer, x[:, at:at + N], at)[0]
        return _out(layer, _attend(q, *(t.to(q.dtype) for t in kv), layer.scale,
                                   seen_of(B, N, at + N, layer.window, layer.sinks)[:, None]))

    with torch.no_grad():
        near = [reference(layer, x, a, n, kv) for a, n, _, kv in got]
        layer.double()
        want = [reference(layer, x.double(), a, n, kv) for a, n, _, kv in got]
        # what the cache holds is the keys and values to one rounding in 8 bits: half a step of
        # 2^-4, or of the smallest step, 2^-9 of a scale that is 2^-8 of the largest at most
        _, k, v = _split_ref(layer, x[:, :at].double())
        for a, b in zip(got[-1][3], (k, v)):
            size = b.abs().amax()
            assert bool(((a.double() - b).abs() <= b.abs() * 2.0 ** -4 * 1.001 + size * 2.0 ** -17).all())
    for (_, _, a, _), b, c in zip(got, near, want):
        size = float(c.abs().max())
        off, ref = float((a.double() - c).abs().max()), float((b.double() - c).abs().max())
        assert off <= 8 * ref + 1e-5 * size, (off, ref, size)


def test_decoding_of_ragged_chunks():
    # sequences of several lengths in one call: as each by itself
    layer = _layer(4, 2, True, True, 50, 2, seed=7)
    x = torch.randn(3, 80, 256, device="cuda")
    cache = api.Cache.new(12, 2)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    n = torch.tensor([80, 0, 37], dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(n)
    first = layer.step(x, cache, table, zero, n)
    then = layer.step(x[:, :3], cache, table, n, torch.tensor([1, 3, 2], dtype=torch.int32, device="cuda"))
    for b, (a, c) in enumerate(((80, 1), (0, 3), (37, 2))):
        one = api.Cache.new(4, 2)
        row, at = table[:1], torch.tensor([a], dtype=torch.int32, device="cuda")
        if a:
            alone = layer.step(x[b:b + 1, :a], one, row, zero[:1])
            torch.testing.assert_close(alone, first[b:b + 1, :a], rtol=0, atol=1e-5 * float(first.abs().max()))
        alone = layer.step(x[b:b + 1, :c], one, row, at)
        torch.testing.assert_close(alone, then[b:b + 1, :c], rtol=0, atol=1e-5 * float(then.abs().max()))


def test_refusals():
    with pytest.raises(ValueError, match="dim"):
        WindowSelfAttention(100, 2)
    with pytest.raises(ValueError, match="kv_heads"):
        WindowSelfAttention(192, 3, 2)
    with pytest.raises(ValueError, match="window"):
        WindowSelfAttention(128, 2, window=0)
    with pytest.raises(ValueError, match="sinks"):
        WindowSelfAttention(128, 2, sinks=-1)
