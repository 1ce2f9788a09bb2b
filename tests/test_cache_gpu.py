"""The paged 8-bit cache on the GPU: stored bytes, scales and loaded values equal to
those of the definition (tests/cache_ref.py), the attention within bounds from
counted roundings, over chunks, page borders, windows, types and layouts; bad tables;
streams, graphs and repeated calls; all of it together with the attention over a window."""
import ctypes
import math

import pytest
import torch

from cache_ref import PAGE, Pages, attend
from window_ref import check, seen_of
from window_ref import window as window_attend
from sparse_head_self_gb300 import _native, api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def _ids(s):
    return "x".join(map(str, s))


def _int32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rand(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _states(g, B, Hkv, N, dtype, layout="bnhd"):
    if layout == "bhnd":
        return tuple(_rand(g, B, Hkv, N, 64, dtype=dtype) for _ in range(2))
    if layout == "wide":
        return tuple(_rand(g, B, Hkv, N, 104, dtype=dtype)[..., 16:80] for _ in range(2))
    kv = _rand(g, B, N, 2, Hkv, 64, dtype=dtype)
    return kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)


def _cache(pages, Hkv, junk=True, seed=0):
    """A cache full of what earlier use left: any bytes, NaN among them, and scales that mean nothing."""
    cache = api.Cache.new(pages, Hkv)
    if junk:
        g = torch.Generator(device="cuda").manual_seed(seed)
        cache.data.copy_(torch.randint(0, 256, cache.data.shape, generator=g, device="cuda", dtype=torch.uint8))
        cache.scales.copy_(2.0 ** torch.randint(-120, 120, cache.scales.shape, generator=g, device="cuda").float())
        cache.scales.view(-1)[::7] = math.nan
    return cache


def _table(B, M, pages, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[:B * M].to(torch.int32).view(B, M).cuda()


def _same(cache, pages):
    assert torch.equal(cache.data.cpu(), pages.data)
    a, b = cache.scales.cpu(), pages.scales
    assert torch.equal(a.nan_to_num(-1.0), b.nan_to_num(-1.0))


def _error():
    torch.cuda.synchronize()
    code = ctypes.c_uint(0)
    _native.check(_native.lib().fibatt_device_error(1, ctypes.byref(code)))
    return code.value


@TYPES
@pytest.mark.parametrize("layout", ["bnhd", "bhnd", "wide"])
def test_stored_chunk_by_chunk(dtype, layout):
    # chunks that begin, continue and end pages, single tokens among them, tokens of growing and
    # of falling size, a sequence that goes back, one that has no tokens in a call
    g = torch.Generator(device="cuda").manual_seed(1)
    B, Hkv, M = 3, 2, 5
    cache, table = _cache(B * M + 2, Hkv), _table(B, M, B * M + 2)
    pages = Pages(*cache)
    start = torch.zeros(B, dtype=torch.int64)
    for turn, N in enumerate([70, 1, 1, 57, 64, 3, 1, 40]):
        count = torch.tensor([N, max(0, N - 2), N // 2])
        if turn == 6:
            start[0] -= 30
        K, V = _states(g, B, Hkv, N, dtype, layout)
        size = [1.0, 0.5, 4.0, 1e-3, 30.0, 100.0, 1e-2, 1.0][turn]
        K, V = K * size, V / size
        s, n = start.to(torch.int32).cuda(), count.to(torch.int32).cuda()
        api.cache_store(cache, table, K, V, s, n)
        pages.store(table.cpu(), K, V, start, count)
        _same(cache, pages)
        start += count
    for dt in (F32, BF16):
        for first, N in (((0, 0, 0), 200), ((5, 64, 33), 100)):
            n = (start - torch.tensor(first)).clamp(max=N)
            got = api.cache_load(cache, table, N, _int32(*first), n.to(torch.int32).cuda(), dtype=dt)
            want = pages.load(table.cpu(), N, first, n)
            for a, b in zip(got, want):
                assert a.dtype == dt and torch.equal(a.double().cpu(), b)


@TYPES
def test_stored_at_once_and_token_by_token(dtype):
    # the scales agree; bytes differ only where a scale was raised after a token below its smallest normal step
    g = torch.Generator(device="cuda").manual_seed(2)
    K, V = _states(g, 2, 3, 130, dtype)
    once, each = _cache(6, 3), _cache(6, 3)
    table = _table(2, 3, 6)
    api.cache_store(once, table, K, V)
    pages = Pages(*each)
    for n in range(130):
        at = _int32(n, n)
        api.cache_store(each, table, K[:, :, n:n + 1], V[:, :, n:n + 1], at)
        pages.store(table.cpu(), K[:, :, n:n + 1], V[:, :, n:n + 1], (n, n))
    _same(each, pages)
    assert torch.equal(once.scales, each.scales)
    for a, b, x in zip(api.cache_load(once, table, 130, dtype=F32), api.cache_load(each, table, 130, dtype=F32), (K, V)):
        x = x.float()
        # one rounding: half a step, 2^-4 of a value or half the smallest step; two of them token by token
        small = once.scales.max() * 2.0 ** -10
        assert bool(((a - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, small)).all())
        assert bool(((b - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, 2 * small)).all())


@TYPES
def test_values_on_every_border(dtype):
    # ties, the largest, zeros of both signs, the smallest steps, infinities and NaN, the types' extremes
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    ties = (v[1:] + v[:-1]) / 2
    x = torch.cat([v, ties, -v, -ties, torch.tensor([0.0, -0.0, 448.0, -448.0])])
    x = torch.nn.functional.pad(x, (0, -len(x) % 64)).view(-1, 64)
    for top in (448.0, 449.0, 450.0, 1.0, 1.75, 1.7578125, 0.0, 1e-30, 1e-38, 3e38):
        for odd in (0.0, math.inf, -math.inf, math.nan):
            rows = (x * (top / 448.0)).to(dtype)
            K = rows[None, None].cuda().contiguous()
            K[0, 0, 1, 2] = odd
            V = (-K).flip(2).contiguous()
            cache, table = _cache(1, 1, junk=False), _table(1, 1, 1)
            pages = Pages(*cache)
            api.cache_store(cache, table, K, V)
            pages.store(table.cpu(), K, V)
            _same(cache, pages)
            for a, b in zip(api.cache_load(cache, table, K.shape[2], dtype=F32), pages.load(table.cpu(), K.shape[2])):
                assert torch.equal(a.double().cpu().nan_to_num(-7.0), b.float().double().nan_to_num(-7.0)), (top, odd)


def _filled(g, B, Hkv, lens, M, dtype, spare=3, size=1.0):
    """A cache that holds `lens` tokens of each sequence, its table, and those tokens as values in 64 bits."""
    cache, table = _cache(B * M + spare, Hkv), _table(B, M, B * M + spare)
    N = max(max(lens), 1)
    K, V = _states(g, B, Hkv, N, dtype)
    dims = torch.exp(0.5 * _rand(g, Hkv, 1, 64)) * size
    api.cache_store(cache, table, (K * dims).to(dtype), (V * dims).to(dtype), None, _int32(*lens))
    for b, n in enumerate(lens):       # entries that nobody needs
        table[b, (n + PAGE - 1) // PAGE:] = -1 if b % 2 else 2 ** 31 - 1
    k, v = (t.double() for t in api.cache_load(cache, table, N, None, _int32(*lens), dtype=F32))
    return cache, table, k, v


def _check_fwd(q, cache, table, k, v, lens, scale=0.125, window=None, sinks=0, count=None):
    """The queries are those of each sequence's last tokens."""
    N = q.shape[2]
    n = [N] * len(lens) if count is None else count
    start = [a - b for a, b in zip(lens, n)]
    got = api.cache_fwd(q, cache, table, _int32(*start), scale, window, sinks, None if count is None else _int32(*count))
    seen = seen_of(q.shape[0], N, k.shape[2], window, sinks, _int32(*start), _int32(*lens))
    want = attend(q, k, v, scale, seen)
    check("O", got[0], want["O"])
    check("LSE", got[1], want["LSE"])
    return got


@TYPES
@pytest.mark.parametrize("heads", [(1, 1), (4, 1), (12, 4), (16, 2), (34, 2), (3, 3)], ids=_ids)
@pytest.mark.parametrize("N", [1, 2, 5, 16, 40])
def test_attention(dtype, heads, N):
    Hq, Hkv = heads
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [N, N + 63, 64 * 3, 130 + N, 700]
    cache, table, k, v = _filled(g, 5, Hkv, lens, 12, dtype)
    q = _rand(g, 5, N, Hq, 64, dtype=dtype).transpose(1, 2)
    for window, sinks in ((None, 0), (1, 0), (30, 3), (64, 0), (65, 70), (300, 4), (100, 200)):
        _check_fwd(q, cache, table, k, v, lens, window=window, sinks=sinks)


@TYPES
def test_attention_of_ragged_tokens(dtype):
    # counts from none to all; queries left out hold NaN
    g = torch.Generator(device="cuda").manual_seed(4)
    lens, count = [200, 64, 65, 128, 9], [7, 0, 3, 1, 7]
    cache, table, k, v = _filled(g, 5, 2, lens, 4, dtype)
    q = _rand(g, 5, 6, 7, 64, dtype=dtype)
    for b, n in enumerate(count):
        q[b, :, n:] = math.nan
    for window, sinks in ((None, 0), (50, 2)):
        o, lse = _check_fwd(q, cache, table, k, v, lens, window=window, sinks=sinks, count=count)
        for b, n in enumerate(count):
            assert bool((o[b, :, n:] == 0).all()) and bool((lse[b, :, n:] == -math.inf).all())


@TYPES
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("size", [1e-20, 1.0, 1e15])
def test_scales_and_sizes(dtype, scale, size):
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = [300, 77]
    cache, table, k, v = _filled(g, 2, 2, lens, 5, dtype, size=size)
    q = (_rand(g, 2, 4, 3, 64) / size).to(dtype)
    _check_fwd(q, cache, table, k, v, lens, scale)
    _check_fwd(q, cache, table, k, v, lens, scale, 100, 3)


@TYPES
@pytest.mark.parametrize("N", [1, 6])
def test_large_scores_in_growing_order(dtype, N):
    # each page's maximum is far above the last one's, the pages' scales grow, and the values' fall
    g = torch.Generator(device="cuda").manual_seed(6)
    cache, table = _cache(20, 2), _table(1, 12, 20)
    K, V = _states(g, 1, 2, 700, dtype)
    grow = torch.arange(700, device="cuda")[:, None] / 100.0
    api.cache_store(cache, table, (K.abs() * grow).to(dtype), (V * torch.exp2(-2 * grow)).to(dtype))
    k, v = (t.double() for t in api.cache_load(cache, table, 700, dtype=F32))
    q = (_rand(g, 1, 8, N, 64).abs() * 2).to(dtype)
    _check_fwd(q, cache, table, k, v, [700])


@TYPES
@pytest.mark.parametrize("T", [5000, 33000])
def test_long_sequences(dtype, T):
    g = torch.Generator(device="cuda").manual_seed(7)
    M = (T + 63) // 64
    for B, Hq, Hkv, N in ((1, 4, 1, 1), (3, 4, 2, 2)):
        lens = [T, T // 2, 1 + N][:B]
        cache, table, k, v = _filled(g, B, Hkv, lens, M, dtype)
        q = _rand(g, B, Hq, N, 64, dtype=dtype)
        for window, sinks in ((None, 0), (4000, 4), (100, 900)):
            _check_fwd(q, cache, table, k, v, lens, window=window, sinks=sinks)


@TYPES
def test_more_units_than_the_gpu_holds(dtype):
    g = torch.Generator(device="cuda").manual_seed(8)
    B, Hkv = 90, 8
    lens = [1 + 7 * b for b in range(B)]
    cache, table, k, v = _filled(g, B, Hkv, lens, 10, dtype)
    q = _rand(g, B, 2 * Hkv, 1, 64, dtype=dtype)
    _check_fwd(q, cache, table, k, v, lens)
    _check_fwd(q, cache, table, k, v, lens, window=100, sinks=4)


def test_pages_behind_32_bits():
    # pages more than 2^32 bytes into the cache
    g = torch.Generator(device="cuda").manual_seed(9)
    pages = 600000
    cache = api.Cache.new(pages, 1)
    table = torch.tensor([[pages - 1, 3, pages - 70000]], dtype=torch.int32, device="cuda")
    K, V = _states(g, 1, 1, 150, BF16)
    api.cache_store(cache, table, K, V)
    want = Pages(cache.data[:4], cache.scales[:4])      # the same tokens in a small cache
    want.store(torch.tensor([[0, 1, 2]]), K, V)
    assert torch.equal(cache.data[table[0].long()].cpu(), want.data[:3]) and torch.equal(cache.scales[table[0].long()].cpu(), want.scales[:3])
    k, v = api.cache_load(cache, table, 150, dtype=F32)
    for a, b in zip((k, v), want.load(torch.tensor([[0, 1, 2]]), 150)):
        assert torch.equal(a.double().cpu(), b)
    _check_fwd(_rand(g, 1, 4, 1, 64, dtype=BF16), cache, table, k.double(), v.double(), [150])


@TYPES
def test_a_prefix_that_sequences_share(dtype):
    # two full pages in three tables; each sequence goes on in pages of its own
    g = torch.Generator(device="cuda").manual_seed(10)
    cache = _cache(9, 2)
    table = _int32(*[4, 7, 0, 1, 4, 7, 2, 3, 4, 7, 5, 6]).view(3, 4)
    K, V = _states(g, 1, 2, 128, dtype)
    api.cache_store(cache, table[:1], K, V)
    K2, V2 = _states(g, 3, 2, 50, dtype)
    api.cache_store(cache, table, K2, V2, _int32(128, 128, 128))
    k, v = (t.double() for t in api.cache_load(cache, table, 178, dtype=F32))
    assert torch.equal(k[0, :, :128], k[1, :, :128]) and torch.equal(v[0, :, :128], v[2, :, :128])
    _check_fwd(_rand(g, 3, 4, 2, 64, dtype=dtype), cache, table, k, v, [178, 178, 178])


@TYPES
def test_tables_that_do_not_have_the_pages(dtype):
    # tokens without a page are dropped, load as zeros, are attended by nobody, and are reported
    g = torch.Generator(device="cuda").manual_seed(11)
    B, M, pages = 3, 4, 14
    cache, table = _cache(pages, 2), _table(B, M, pages)
    for b, i, bad in ((0, 1, -1), (1, 0, pages), (2, 3, 2 ** 31 - 1), (2, 1, -2 ** 31)):
        table[b, i] = bad
    before = Pages(*cache)
    K, V = _states(g, B, 2, 256, dtype)
    api.cache_store(cache, table, K, V)
    assert _error() == 16
    before.store(table.cpu(), K, V)
    _same(cache, before)
    k, v = api.cache_load(cache, table, 256, dtype=F32)
    assert _error() == 16
    for a, b in zip((k, v), before.load(table.cpu(), 256)):
        assert torch.equal(a.double().cpu(), b)
    q = _rand(g, B, 4, 2, 64, dtype=dtype)
    got = api.cache_fwd(q, cache, table, _int32(254, 254, 254), 0.125)
    assert _error() == 16
    there = (table >= 0) & (table < pages)
    seen = seen_of(B, 2, 256) & there.repeat_interleave(64, 1)[:, None]
    want = attend(q, k.double(), v.double(), 0.125, seen)
    check("O", got[0], want["O"])
    check("LSE", got[1], want["LSE"])
    # a window that needs none of the missing pages reports nothing
    api.cache_fwd(q[:2], cache, table[:2], _int32(254, 254), 0.125, 60)
    assert _error() == 0


def test_starts_outside_the_table():
    g = torch.Generator(device="cuda").manual_seed(12)
    cache, table = _cache(8, 1), _table(4, 2, 8)
    K, V = _states(g, 4, 1, 40, BF16)
    far = 2 ** 31 - 1
    for start in ((-20, 100, -far - 1, far), (-40, 128, 127, 88)):
        pages = Pages(*cache)
        api.cache_store(cache, table, K, V, _int32(*start))
        assert _error() == 16
        pages.store(table.cpu(), K, V, start)
        _same(cache, pages)
        got = api.cache_load(cache, table, 40, _int32(*start), dtype=F32)
        assert _error() == 16
        for a, b in zip(got, pages.load(table.cpu(), 40, start)):
            assert torch.equal(a.double().cpu().nan_to_num(-7.0), b.float().double().nan_to_num(-7.0))
    # queries before the sequence are padding; those behind the table attend nothing and are reported
    cache, table, k, v = _filled(g, 2, 1, [128, 128], 2, BF16)
    q = _rand(g, 2, 2, 30, 64, dtype=BF16)
    o, lse = api.cache_fwd(q, cache, table, _int32(-25, 110), 0.125)
    assert _error() == 16
    want = attend(q, k, v, 0.125, seen_of(2, 30, 128, None, 0, _int32(-25, 110)))
    check("O", o, want["O"])
    check("LSE", lse, want["LSE"])
    assert bool((o[0, :, :25] == 0).all()) and bool((lse[1, :, 18:] == -math.inf).all())


@TYPES
def test_a_tokens_nan_reaches_those_who_attend_it(dtype):
    g = torch.Generator(device="cuda").manual_seed(13)
    cache, table = _cache(8, 2), _table(2, 4, 8)
    K, V = (t.contiguous() for t in _states(g, 2, 2, 200, dtype, "bhnd"))
    clean = api.Cache(cache.data.clone(), cache.scales.clone())
    api.cache_store(clean, table, K, V)
    V[0, 0, 70, 5] = math.nan
    api.cache_store(cache, table, K, V)
    q = _rand(g, 2, 4, 1, 64, dtype=dtype)
    at = _int32(199, 199)
    want, got = api.cache_fwd(q, clean, table, at, 0.125)[0], api.cache_fwd(q, cache, table, at, 0.125)[0]
    assert bool(got[0, :2, :, 5].isnan().all())
    got[0, :2, :, 5] = want[0, :2, :, 5]
    assert torch.equal(got, want)
    # one place behind the NaN, a window away from it
    assert torch.equal(*(api.cache_fwd(q, c, table, at, 0.125, 129)[0] for c in (clean, cache)))


@TYPES
def test_only_the_results_rows_are_written(dtype):
    g = torch.Generator(device="cuda").manual_seed(14)
    lens = [100, 64]
    cache, table, k, v = _filled(g, 2, 2, lens, 3, dtype)

    def inside(H, N):
        big = torch.full((2, N + 5, H + 2, 80), 77.0, dtype=dtype, device="cuda")
        return big, big[:, 2:2 + N, 1:1 + H, 8:72].transpose(1, 2)

    q = _rand(g, 2, 4, 3, 64, dtype=dtype)
    bigs = [inside(4, 3), inside(2, 70), inside(2, 70)]
    api.cache_fwd(q, cache, table, _int32(97, 61), 0.125, O=bigs[0][1])
    want = [api.cache_fwd(q, cache, table, _int32(97, 61), 0.125)[0]]
    n = _int32(60, 34)
    api.cache_load(cache, table, 70, _int32(40, 30), n, K=bigs[1][1], V=bigs[2][1])
    want += api.cache_load(cache, table, 70, _int32(40, 30), n, dtype=dtype)
    for (big, view), x in zip(bigs, want):
        assert torch.equal(view, x)
        view.fill_(77.0)
        assert bool((big == 77.0).all())


@TYPES
def test_streams_and_two_calls_at_once(dtype):
    g = torch.Generator(device="cuda").manual_seed(15)
    sets = [(*_filled(g, 2, 2, [700, 333], 11, dtype)[:2], _rand(g, 2, 8, 1, 64, dtype=dtype)) for _ in range(2)]
    at = _int32(699, 332)
    want = [api.cache_fwd(q, cache, table, at, 0.125) for cache, table, q in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(5):
        for i, (s, (cache, table, q)) in enumerate(zip(streams, sets)):
            got[i].append(api.cache_fwd(q, cache, table, at, 0.125, stream=s))
    torch.cuda.synchronize()
    for w, rs in zip(want, got):
        for r in rs:
            assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])


@TYPES
def test_captured_and_replayed_token_by_token(dtype):
    # one graph stores a token, attends and moves on: starts, tables and tokens are read on the device
    g = torch.Generator(device="cuda").manual_seed(16)
    B, Hq, Hkv, M = 2, 8, 2, 4
    cache, table = _cache(B * M, Hkv), _table(B, M, B * M)
    K, V = (t.contiguous() for t in _states(g, B, Hkv, 150, dtype))
    Q = _rand(g, B, Hq, 150, 64, dtype=dtype)
    api.cache_store(cache, table, K[:, :, :60], V[:, :, :60])
    pages = Pages(*cache)
    q, k, v = (t[:, :, :1].clone() for t in (Q, K, V))
    at = _int32(60, 60)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):       # (stores nothing new: the token before)
        api.cache_store(cache, table, K[:, :, 59:60], V[:, :, 59:60], at - 1)
        api.cache_fwd(q, cache, table, at - 1, 0.125, 40, 2)
    torch.cuda.synchronize()
    pages.store(table.cpu(), K[:, :, 59:60], V[:, :, 59:60], (59, 59))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_store(cache, table, k, v, at)
        o, lse = api.cache_fwd(q, cache, table, at, 0.125, 40, 2)
        at += 1
    for n in range(60, 150):
        for t, src in ((q, Q), (k, K), (v, V)):
            t.copy_(src[:, :, n:n + 1])
        graph.replay()
        pages.store(table.cpu(), K[:, :, n:n + 1], V[:, :, n:n + 1], (n, n))
        if n % 16 == 0 or n == 149:
            kk, vv = (t.cuda() for t in pages.load(table.cpu(), n + 1))
            want = attend(q, kk, vv, 0.125, seen_of(B, 1, n + 1, 40, 2))
            check("O", o, want["O"])
            check("LSE", lse, want["LSE"])
    _same(cache, pages)
    assert at.tolist() == [150, 150]


@TYPES
def test_the_same_result_on_every_call(dtype):
    g = torch.Generator(device="cuda").manual_seed(17)
    cache, table, _, _ = _filled(g, 3, 2, [2000, 900, 64], 32, dtype)
    q = _rand(g, 3, 8, 2, 64, dtype=dtype)
    at = _int32(1998, 898, 62)
    first = api.cache_fwd(q, cache, table, at, 0.125)
    for _ in range(4):
        again = api.cache_fwd(q, cache, table, at, 0.125)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@TYPES
def test_a_prompt_in_chunks_and_then_tokens(dtype):
    # the first chunk attends itself, the next what the cache gives back and itself, tokens and a
    # few tokens the cache: each against the definition on the values that the cache holds
    g = torch.Generator(device="cuda").manual_seed(18)
    B, Hq, Hkv, M, window, sinks = 2, 8, 2, 8, 100, 3
    cache, table = _cache(B * M, Hkv), _table(B, M, B * M)
    pages = Pages(*cache)
    at = 0
    for N in (150, 90, 1, 1, 5, 1):
        K, V = _states(g, B, Hkv, N, dtype)
        q = _rand(g, B, Hq, N, 64, dtype=dtype)
        start = _int32(at, at)
        api.cache_store(cache, table, K, V, start)
        pages.store(table.cpu(), K, V, (at, at))
        seen = seen_of(B, N, at + N, window, sinks)
        kk, vv = (t.cuda() for t in pages.load(table.cpu(), at + N))
        if N > 16:
            k, v = api.cache_load(cache, table, at + N, dtype=dtype)
            assert torch.equal(k.double(), kk) and torch.equal(v.double(), vv)
            got, want = api.window_fwd(q, k, v, 0.125, window, sinks), window_attend(q, kk, vv, 0.125, seen)
        else:
            got, want = api.cache_fwd(q, cache, table, start, 0.125, window, sinks), attend(q, kk, vv, 0.125, seen)
        check("O", got[0], want["O"])
        check("LSE", got[1], want["LSE"])
        at += N


def test_gpu_refusals():
    g = torch.Generator(device="cuda").manual_seed(19)
    cache, table = _cache(4, 2), _table(2, 2, 4)
    K, V = _states(g, 2, 2, 5, BF16)
    q = _rand(g, 2, 4, 1, 64, dtype=BF16)
    with pytest.raises(ValueError, match="table"):
        api.cache_store(cache, table[:1], K, V)
    with pytest.raises(ValueError, match="dtype"):
        api.cache_store(cache, table.long(), K, V)
    with pytest.raises(ValueError, match="start"):
        api.cache_store(cache, table, K, V, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="count"):
        api.cache_store(cache, table, K, V, None, _int32(1))
    with pytest.raises(ValueError, match="K has shape"):
        api.cache_store(cache, table, K[:, :1], V[:, :1])
    with pytest.raises(ValueError, match="V has"):
        api.cache_store(cache, table, K, V.float())
    with pytest.raises(ValueError, match="data"):
        api.cache_store(api.Cache(cache.data[..., :64], cache.scales), table, K, V)
    with pytest.raises(ValueError, match="scales"):
        api.cache_store(api.Cache(cache.data, cache.scales[:3]), table, K, V)
    with pytest.raises(ValueError, match="data"):
        api.cache_load(api.Cache(cache.data.view(torch.int8), cache.scales), table, 5)
    with pytest.raises(ValueError, match="dtype"):
        api.cache_load(cache, table, 5, dtype=torch.float16)
    with pytest.raises(api.FibattError, match=">= 1"):
        api.cache_load(cache, table, 0)
    with pytest.raises(api.FibattError, match="divide"):
        api.cache_fwd(q[:, :3], cache, table, None, 0.125)
    with pytest.raises(api.FibattError, match="window"):
        api.cache_fwd(q, cache, table, None, 0.125, 0)
    with pytest.raises(ValueError, match="CUDA"):
        api.cache_fwd(q, api.Cache(cache.data.cpu(), cache.scales.cpu()), table, None, 0.125)
