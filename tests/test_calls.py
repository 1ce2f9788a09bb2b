"""The short way from Python into the library (binding/calls.cpp): it takes the calls of
the usual form and gives what the general way gives; every other form, and every
call that is to be refused, it leaves alone."""
import math

import pytest
import torch

from sparse_head_self_gb300 import _native, api
from sparse_head_self_gb300.build import build_all

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("window_fwd", "window_bwd", "cache_store", "cache_load", "cache_fwd")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_all()
    yield


def test_forms_that_it_does_not_take():
    calls = _native.calls()
    q, n = torch.zeros(1, 2, 3, 64), torch.zeros(1, dtype=torch.int32)
    data, scales = api.Cache.new(2, 2, "cpu")
    odd = (None, 3, "q", [q], q, n, object(), q.numpy(), torch.nn.Parameter(q), q.to_sparse(), torch.zeros(0))
    for name in NAMES:
        f = getattr(calls, name)
        for count in range(13):       # any number of arguments, of any kind
            for x in odd:
                assert f(*([x] * count)) is None, (name, count, x)
    assert calls.window_fwd(q, q, q, 0.125, None, 0, None, None) is None        # not on a GPU
    assert calls.window_bwd(q, q, q, q, q[..., 0], q, 0.125, None, 0, None, None) is None
    assert calls.cache_store(data, scales, n[:, None], q, q, None, None) is None
    assert calls.cache_load(data, scales, n[:, None], 3, None, None, False) is None
    assert calls.cache_fwd(q, data, scales, n[:, None], None, 0.125, None, 0, None) is None


def test_addresses_are_checked():
    calls = _native.calls()
    with pytest.raises(TypeError):
        calls.use(1, 2)
    with pytest.raises(ValueError):
        calls.use(1, 2, 3, 4, 5, 0)
    with pytest.raises(TypeError):
        calls.use(1, 2, 3, 4, 5, "6")
    _native.calls()


def _inputs(dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, do = (torch.randn(2, 50, 4, 64, generator=g, device="cuda").to(dtype).transpose(1, 2) for _ in range(2))
    kv = torch.randn(2, 90, 2, 2, 64, generator=g, device="cuda").to(dtype)
    return q, kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2), do


def _int32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_both_ways_give_the_same(dtype, monkeypatch):
    taken = []
    calls = _native.calls()

    class Watched:
        def __getattr__(self, name):
            def call(*a):
                r = getattr(calls, name)(*a)
                taken.append((name, r is not None))
                return r
            return call

    monkeypatch.setattr(api, "_calls", Watched())
    here = torch.cuda.current_stream()
    q, k, v, do = _inputs(dtype)
    for window, sinks in ((None, 0), (20, 3), (10 ** 12, 10 ** 12)):
        for start, n in ((None, None), (_int32(40, 3), _int32(90, 41))):
            how = (window, sinks, start, n)
            o, lse = api.window_fwd(q, k, v, 0.125, *how)
            want = api.window_fwd(q, k, v, 0.125, *how, stream=here)
            got = [o, lse, *api.window_bwd(q, k, v, o, lse, do, 0.125, *how)]
            want += api.window_bwd(q, k, v, o, lse, do, 0.125, *how, stream=here)
            for a, b in zip(got, want):
                assert torch.equal(a, b) and a.stride() == b.stride() and a.dtype == b.dtype
    table, start, count = _int32(3, 1, 0, 2).view(2, 2), _int32(7, 30), _int32(90, 33)
    caches = [api.Cache.new(4, 2) for _ in range(2)]
    for cache, stream in zip(caches, (None, here)):
        api.cache_store(cache, table, k, v, start, count, stream=stream)
    for a, b in zip(*caches):
        assert torch.equal(a, b)
    for a, b in zip(api.cache_load(caches[0], table, 90, start, count, dtype), api.cache_load(caches[0], table, 90, start, count, dtype, stream=here)):
        assert torch.equal(a, b) and a.stride() == b.stride() and a.dtype == dtype
    for n in (None, _int32(50, 3)):
        a = api.cache_fwd(q, caches[0], table, start, 0.125, 20, 2, n)
        b = api.cache_fwd(q, caches[0], table, start, 0.125, 20, 2, n, stream=here)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[0].stride() == b[0].stride()
    assert all(ok for _, ok in taken) and {name for name, _ in taken} == set(NAMES)
    # forms that go the general way: results given, a scale that is no float, gradients on another stream
    taken.clear()
    api.window_fwd(q, k, v, 1, 20)
    assert taken == [("window_fwd", False)]
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_refusals_are_the_general_ways(monkeypatch):
    q, k, v, do = _inputs(BF16)
    with pytest.raises(api.FibattError, match="window"):
        api.window_fwd(q, k, v, 0.125, 0)
    with pytest.raises(api.FibattError, match="window"):
        api.window_fwd(q, k, v, 0.125, -1)
    with pytest.raises(api.FibattError, match="sinks"):
        api.window_fwd(q, k, v, 0.125, 3, -1)
    with pytest.raises(api.FibattError, match="scale"):
        api.window_fwd(q, k, v, math.nan, 3)
    with pytest.raises(api.FibattError, match="16-byte"):
        api.window_fwd(torch.zeros(2, 4, 50, 65, dtype=BF16, device="cuda")[..., 1:], k, v, 0.125)
    o, lse = api.window_fwd(q, k, v, 0.125)
    with pytest.raises(ValueError, match="LSE"):
        api.window_bwd(q, k, v, o, lse[:, :1], do, 0.125)
    with pytest.raises(ValueError, match="dO"):
        api.window_bwd(q, k, v, o, lse, do[:, :1], 0.125)
    monkeypatch.setenv("FIBATT_FAULT", "launch")
    cache, table = api.Cache.new(4, 2), _int32(0, 1, 2, 3).view(2, 2)
    for call in (lambda: api.window_fwd(q, k, v, 0.125), lambda: api.window_bwd(q, k, v, o, lse, do, 0.125),
                 lambda: api.cache_store(cache, table, k, v), lambda: api.cache_load(cache, table, 9),
                 lambda: api.cache_fwd(q, cache, table, None, 0.125)):
        with pytest.raises(api.FibattError, match="injected"):
            call()


@pytest.mark.gpu
def test_a_stream_of_the_threads_own():
    q, k, v, _ = _inputs(BF16, 3)
    want = api.window_fwd(q, k, v, 0.125, 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = api.window_fwd(q, k, v, 0.125, 20)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
