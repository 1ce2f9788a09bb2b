"""Calls of the window attention and the cache that the short way (binding/calls.cpp) leaves to the general one:
with results or a workspace given, on a stream that is named, with a scale that is no float.  The
tensors given are those that are written and returned, with the short way's values."""
import pytest
import torch

from test_calls import _inputs, _int32
from sparse_head_self_gb300 import _native, api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def watched(monkeypatch):
    """Names of the calls that went the short way."""
    taken, calls = [], _native.calls()

    class Watched:
        def __getattr__(self, name):
            def call(*a):
                r = getattr(calls, name)(*a)
                if r is not None:
                    taken.append(name)
                return r
            return call

    monkeypatch.setattr(api, "_calls", Watched())
    return taken


def _equal(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_results_that_are_given(dtype, watched):
    q, k, v, do = _inputs(dtype)
    how = (0.125, 20, 3, _int32(40, 3), _int32(90, 41))
    O, LSE = api.window_fwd(q, k, v, *how)
    grads = api.window_bwd(q, k, v, O, LSE, do, *how)
    table, start, count = _int32(3, 1, 0, 2).view(2, 2), _int32(7, 30), _int32(90, 33)
    cache = api.Cache.new(4, 2)
    api.cache_store(cache, table, k, v, start, count)
    loaded = api.cache_load(cache, table, 90, start, count, dtype)
    attended = api.cache_fwd(q, cache, table, start, 0.125, 20, 2)
    assert watched == ["window_fwd", "window_bwd", "cache_store", "cache_load", "cache_fwd"]
    watched.clear()
    other = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    for names, call, want in (
            (("O", "LSE"), lambda **x: api.window_fwd(q, k, v, *how, **x), (O, LSE)),
            (("dQ", "dK", "dV"), lambda **x: api.window_bwd(q, k, v, O, LSE, do, *how, **x), grads),
            (("K", "V"), lambda **x: api.cache_load(cache, table, 90, start, count, dtype, **x), loaded),
            (("O", "LSE"), lambda **x: api.cache_fwd(q, cache, table, start, 0.125, 20, 2, **x), attended)):
        for given in [(n,) for n in names] + [names]:
            mine = {n: other(want[names.index(n)]) for n in given}
            got = call(**mine)
            _equal(got, want)
            for n in given:
                assert got[names.index(n)].data_ptr() == mine[n].data_ptr(), n
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    _equal(api.window_bwd(q, k, v, O, LSE, do, *how, workspace=ws), grads)
    if dtype == BF16:
        assert not bool((ws == 255).all())
    assert watched == []


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_streams_that_are_named(dtype, watched):
    q, k, v, do = _inputs(dtype)
    table, start = _int32(3, 1, 0, 2).view(2, 2), _int32(7, 30)
    caches = [api.Cache.new(4, 2) for _ in range(2)]
    want, got = [], []
    side = torch.cuda.Stream()
    for cache, stream, to in ((caches[0], None, want), (caches[1], side, got)):
        torch.cuda.synchronize()
        to += api.window_fwd(q, k, v, 0.125, 20, stream=stream)
        to += api.window_bwd(q, k, v, *to, do, 0.125, 20, stream=stream)
        api.cache_store(cache, table, k, v, start, stream=stream)
        to += api.cache_load(cache, table, 90, start, dtype=dtype, stream=stream)
        to += api.cache_fwd(q, cache, table, start, 0.125, 20, stream=stream)
    torch.cuda.synchronize()
    _equal(got, want)
    _equal(caches[0], caches[1])
    assert len(watched) == 5      # of the calls without a stream


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_scale_that_is_no_float(dtype, watched):
    q, k, v, do = _inputs(dtype)
    want = api.window_fwd(q, k, v, 1.0, 20)
    want += api.window_bwd(q, k, v, *want, do, 1.0, 20)
    table, cache = _int32(3, 1, 0, 2).view(2, 2), api.Cache.new(4, 2)
    api.cache_store(cache, table, k, v)
    want += api.cache_fwd(q, cache, table, None, 1.0)
    watched.clear()
    for one in (1, torch.tensor(1.0)):
        got = api.window_fwd(q, k, v, one, 20)
        got += api.window_bwd(q, k, v, *got, do, one, 20)
        got += api.cache_fwd(q, cache, table, None, one)
        _equal(got, want)
    assert watched == []
