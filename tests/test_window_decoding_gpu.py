"""Decoding with the decoder's self-attention layer where callers' tensors are of several
types, tables end near the tokens, and calls are captured."""
import pytest
import torch

from test_cache_gpu import _error
from sparse_head_self_gb300 import api
from sparse_head_self_gb300.block import WindowSelfAttention

pytestmark = pytest.mark.gpu


def _layer(dim, heads, kv_heads, places, **how):
    torch.manual_seed(0)
    return WindowSelfAttention(dim, heads, kv_heads, norm=True, rotary=api.rotary_angles(places, 32), **how).cuda()


def _table(B, M):
    return torch.arange(B * M, dtype=torch.int32, device="cuda").view(B, M)


@pytest.mark.parametrize("N", [2, 100])
def test_a_step_in_mixed_precision(N):
    # keys and values are of the layer's compute type, whatever x's is
    layer = _layer(256, 4, 2, 400, window=50, sinks=2)
    x = torch.randn(2, N, 256, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    with torch.autocast("cuda", dtype=torch.bfloat16):
        got = layer.step(x, api.Cache.new(4, 2), _table(2, 2), start)
        want = layer(x).detach()
    assert got.dtype is torch.bfloat16 and bool(got.isfinite().all())
    # 8-bit keys and values: a key's 2^-4 moves a weight, a value's its sum; outputs within a tenth of their size
    off = (got.float() - want.float()).norm() / want.float().norm()
    assert float(off) < 0.1, float(off)


@pytest.mark.parametrize("N", [5, 40])
def test_left_out_tokens_behind_the_table_of_angles(N):
    # a chunk's last tokens do not count: their places may lie behind the table's
    layer = _layer(256, 4, 2, 64, window=30, sinks=2)
    x = torch.randn(3, 64 + N, 256, device="cuda")
    cache, table = api.Cache.new(6, 2), _table(3, 2)
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    at = torch.tensor([62, 0, 60], dtype=torch.int32, device="cuda")
    layer.step(x[:, :62], cache, table, zero, at)
    count = torch.tensor([2, 0, N + 9], dtype=torch.int32, device="cuda").clamp(max=4)
    got = layer.step(x[:, 62:62 + N], cache, table, at, count)
    torch.cuda.synchronize()
    assert _error() == 0
    one = api.Cache.new(2, 2)
    layer.step(x[:1, :62], one, table[:1], zero[:1])
    alone = layer.step(x[:1, 62:64], one, table[:1], at[:1])
    torch.testing.assert_close(got[:1, :2], alone, rtol=0, atol=1e-5 * float(got.abs().max()))


def test_a_captured_step():
    layer = _layer(256, 4, 2, 400, window=50, sinks=2)
    cache, table = api.Cache.new(8, 2), _table(2, 4)
    other = api.Cache.new(8, 2)
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 1, 256, device="cuda")
    layer.step(x, other, table, start)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer.step(x, cache, table, start)
        start += 1
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    for t in range(130):
        x.copy_(torch.randn(2, 1, 256, device="cuda"))
        g.replay()
        want = layer.step(x, other, table, at)
        at += 1
        assert torch.equal(got, want), t
    assert torch.equal(cache.data, other.data) and torch.equal(cache.scales, other.scales)
