"""The decoder layer's step where it takes many tokens at once, page by page and from loaded tokens: it needs the
pages of the window and of the sinks alone, whatever the table has elsewhere; its scratch does not grow with
the table of a layer with a window; starts, lengths and windows in every order against the definition."""
import pytest
import torch

from test_cache_gpu import _error
from test_layers_gpu import _attend
from test_window_layer_gpu import _layer, _out, _split_ref
from window_ref import check, seen_of, window
from sparse_head_self_gb300 import api
from sparse_head_self_gb300.block import WindowSelfAttention

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(params=[None, True, False], ids=["rule", "pages", "loaded"])
def way(request, monkeypatch):
    """As the layer's rule has it, and each of the two ways."""
    if request.param is not None:
        monkeypatch.setattr(WindowSelfAttention, "_page_by_page", lambda *a: request.param)
    return request.param


def _int32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _fill(layer, x, cache, table, lens):
    """The first lens[b] tokens of every sequence."""
    zero = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    layer.step(x, cache, table, zero, _int32(*lens))


@pytest.mark.parametrize("N", [3, 40, 70, 300])
@pytest.mark.parametrize("window,sinks", [(90, 3), (64, 0), (200, 70), (1, 1)])
def test_pages_behind_the_window_may_be_given_back(N, window, sinks, way):
    layer = _layer(4, 1, True, False, window, sinks, seed=11)
    B, M = 3, 20
    lens = (700, 200, 900)
    x = torch.randn(B, 900, 256, device="cuda")
    more = torch.randn(B, N, 256, device="cuda")
    got = []
    for given_back in (False, True):
        cache = api.Cache.new(B * M, 1)
        table = torch.arange(B * M, dtype=torch.int32, device="cuda").view(B, M)
        _fill(layer, x, cache, table, lens)
        if given_back:
            for b, n in enumerate(lens):
                first, last = (sinks + 63) // 64, max(0, n - window + 1) // 64
                table[b, first:last] = -1 if b % 2 else 2 ** 31 - 1
                table[b, (n + N + 63) // 64:] = -5
        assert _error() == 0
        got.append(layer.step(more, cache, table, _int32(*lens)))
        assert _error() == 0
    assert torch.equal(*got)


@pytest.mark.parametrize("band", [(None, 0), (90, 3), (700, 3), (3000, 0)], ids=str)
@pytest.mark.parametrize("N", [2, 150])
def test_sequences_without_tokens_need_no_pages(band, N, way):
    layer = _layer(4, 1, False, True, *band, seed=13)
    B, M = 3, 8
    cache = api.Cache.new(M, 1)
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    table[1] = torch.arange(M)
    x = torch.randn(B, N, 256, device="cuda")
    out = layer.step(x, cache, table, _int32(100, 0, 0), _int32(0, N, 0))
    assert _error() == 0
    other = api.Cache.new(M, 1)
    alone = layer.step(x[1:2], other, table[1:2], _int32(0))
    torch.testing.assert_close(out[1:2], alone, rtol=0, atol=1e-5 * float(alone.abs().max()))
    assert torch.equal(out[0], layer.proj.bias.expand_as(out[0])) and torch.equal(out[2], out[0])


def test_scratch_does_not_grow_with_the_table(way):
    layer = WindowSelfAttention(256, 4, 4, window=100, sinks=4).cuda()
    x = torch.randn(2, 600, 256, device="cuda")
    cache = api.Cache.new(64, 4)
    table = torch.full((2, 4096), -1, dtype=torch.int32, device="cuda")
    table[:, :32] = torch.arange(64).view(2, 32)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for n in (600, 300):
        layer.step(x[:, :n], cache, table, _int32(0, 0) if n == 600 else _int32(600, 600))
    torch.cuda.synchronize()
    # keys and values of 704 tokens at most are 2.9 MB, the projection's and the attention's results 4.9
    assert torch.cuda.max_memory_allocated() - before < 32e6


@pytest.mark.parametrize("kv_heads,rot", [(4, True), (1, False)])
@pytest.mark.parametrize("band", [(None, 0), (1, 0), (64, 0), (100, 30), (30, 100), (130, 1), (500, 4), (2, 600)], ids=str)
@pytest.mark.parametrize("N", [33, 130, 257])
def test_starts_and_lengths_against_the_definition(kv_heads, rot, band, N, way):
    layer = _layer(4, kv_heads, True, rot, *band, seed=17)
    lens = (0, 20, 64, 99, 128, 129) if rot else (0, 20, 99, 128, 400, 611)
    B, M = len(lens), 15
    cache = api.Cache.new(B * M, kv_heads)
    table = torch.randperm(B * M, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, M).cuda()
    x = torch.randn(B, max(lens) + N, 256, device="cuda")
    _fill(layer, x[:, :max(lens)], cache, table, lens)
    more = torch.stack([x[b, n:n + N] for b, n in enumerate(lens)])
    count = (N, N - 5, N, 1, N, N // 2)
    out = layer.step(more, cache, table, _int32(*lens), _int32(*count))
    assert _error() == 0
    kv = api.cache_load(cache, table, max(lens) + N, None, _int32(*lens) + _int32(*count), dtype=torch.float32)
    layer.double()
    with torch.no_grad():
        for b, (n, c) in enumerate(zip(lens, count)):
            q = _split_ref(layer, more[b:b + 1].double(), n)[0][:, :, :c]
            want = _out(layer, _attend(q, *(t[b:b + 1, :, :n + c].double() for t in kv), layer.scale,
                                       seen_of(1, c, n + c, layer.window, layer.sinks)[:, None]))
            size = float(want.abs().max())
            # 32-bit arithmetic throughout: projections of 256 products, 22-bit products and sums in the attention
            torch.testing.assert_close(out[b:b + 1, :c].double(), want, rtol=0, atol=1e-5 * size)
            assert torch.equal(out[b, c:], layer.proj.bias.float().expand_as(out[b, c:]))


@pytest.mark.parametrize("band", [(None, 0), (90, 3)], ids=str)
def test_tokens_behind_the_table_are_reported(band, way):
    layer = _layer(4, 1, False, False, *band, seed=19)
    cache = api.Cache.new(6, 1)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    x = torch.randn(2, 260, 256, device="cuda")
    out = layer.step(x, cache, table, _int32(0, 10))
    assert _error() == 16
    assert torch.equal(out[1, 182:], layer.proj.bias.expand_as(out[1, 182:]))
    other = api.Cache.new(6, 1)
    alone = layer.step(x[:, :182], other, table, _int32(0, 10))
    assert _error() == 0
    torch.testing.assert_close(out[:, :182], alone, rtol=0, atol=1e-5 * float(alone.abs().max()))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("band", [(None, 0), (1, 0), (64, 0), (100, 30), (30, 100), (130, 1), (500, 4), (2, 600), (1000, 1000)], ids=str)
@pytest.mark.parametrize("N", [40, 200])
def test_attention_to_loaded_tokens(dtype, band, N):
    # the attention alone, in both types, with bounds from counted roundings
    g = torch.Generator(device="cuda").manual_seed(23)
    lens, M, Hkv = (0, 20, 99, 128, 400, 611, 5), 13, 2
    B = len(lens)
    layer = WindowSelfAttention(512, 8, Hkv, *band)
    cache = api.Cache.new(B * M, Hkv)
    table = torch.randperm(B * M, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, M).cuda()
    q = torch.randn(B, N, 8, 64, generator=g, device="cuda").to(dtype).transpose(1, 2)
    K, V = (torch.randn(B, Hkv, 64 * M, 64, generator=g, device="cuda") for _ in range(2))
    start = _int32(*lens)
    held = start + _int32(N, N - 5, N, 1, N, N // 2, 0)
    api.cache_store(cache, table, K, V, None, held)
    k, v = (t.double() for t in api.cache_load(cache, table, 64 * M, None, held, dtype=F32))
    got = layer._attend_loaded(q, cache, table, start, held)
    kv_len = torch.where(held > start, held, 0)       # a sequence without tokens attends nothing
    want = window(q, k, v, 0.125, seen_of(B, N, 64 * M, *band, start, kv_len))
    check("O", got, want["O"])


def test_the_way_that_is_taken():
    # what was measured on both sides (the figures at the rule)
    def pages(B, rows, places, window, dtype=BF16):
        layer = WindowSelfAttention(1024, 16, 4, window, 4 if window else 0)
        return layer._page_by_page(B, rows // 4, places, dtype)

    assert pages(8, 256, 16448, 1024) and not pages(8, 512, 16448, 1024)
    assert pages(8, 128, 16448, None) and not pages(8, 256, 16448, None)
    assert pages(32, 128, 16448, 128) and not pages(32, 192, 16448, 128)
    assert pages(1, 1024, 1600, 128) and not pages(1, 1024, 16448, None)
    assert not pages(1, 4 * 16384, 16448, 4096) and pages(1, 1024, 16448, None, F32)
    assert pages(64, 4, 16448, 1024) and pages(16, 4, 16448, None)


@pytest.mark.parametrize("band", [(None, 0), (90, 3)], ids=str)
def test_captured_and_replayed_chunk_by_chunk(band, way):
    # one graph takes a chunk and moves on, on another stream than the layer's memory came from
    layer = _layer(4, 2, True, True, *band, seed=29)
    B, M, N = 2, 6, 64
    x = torch.randn(B, 5 * N, 256, device="cuda")
    table = torch.randperm(B * M, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, M).cuda()
    plain, cache = (api.Cache.new(B * M, 2) for _ in range(2))
    want = [layer.step(x[:, i * N:(i + 1) * N], plain, table, _int32(i * N, i * N)) for i in range(5)]
    part, at = torch.zeros(B, N, 256, device="cuda"), _int32(0, 0)
    count = _int32(N, N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(part, cache, table, at, count)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = layer.step(part, cache, table, at, count)
            at += count
        for i in range(5):
            part.copy_(x[:, i * N:(i + 1) * N])
            graph.replay()
            torch.testing.assert_close(out, want[i], rtol=0, atol=1e-5 * float(want[i].abs().max()))
    side.synchronize()
    assert at.tolist() == [5 * N, 5 * N]
    for a, b in zip(cache, plain):
        assert torch.equal(a, b)
