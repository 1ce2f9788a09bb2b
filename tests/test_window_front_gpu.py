"""The attention over a window with few sinks where those lie in front of the windows' first
key tiles, on the GPU: values, gradients, layouts, masked places, and the rule that
takes it."""
import math

import pytest
import torch

from test_cross_gpu import _inputs
from test_window_gpu import _check_all, _int32, _ragged, _run, _seen
from window_ref import check, window
from sparse_head_self_gb300 import api

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
SIZES = [(1, 2, 1, 1000, 1000), (2, 4, 2, 391, 391), (2, 6, 2, 700, 1300), (3, 1, 1, 260, 2000), (2, 2, 2, 511, 530)]
BANDS = [(100, 1), (128, 4), (129, 8), (97, 9), (120, 16), (250, 17), (256, 32), (3, 2)]
_ids = lambda s: "x".join(map(str, s))  # noqa: E731


def _fronted(err):
    """Whether the forward calls that FIBATT_PROFILE printed ran the kernel's form for it."""
    lines = [x for x in err.splitlines() if "cross_fwd_mma_kernel" in x]
    assert lines, err
    return ["cross_fwd_mma_kernel<1, true, true," in x for x in lines]


@pytest.mark.parametrize("size,band,want", [((1, 4, 2, 2000, 2000), (128, 4), True), ((1, 4, 2, 2000, 2000), (128, 0), False),
                                            ((1, 4, 2, 2000, 2000), (128, 33), False), ((1, 4, 2, 255, 2000), (128, 4), False),
                                            ((1, 4, 2, 2000, 2000), (None, 4), False)], ids=str)
def test_which_calls_take_it(size, band, want, capfd, monkeypatch):
    q, k, v, _ = _inputs(BF16, *size)
    monkeypatch.setenv("FIBATT_PROFILE", "1")
    capfd.readouterr()
    api.window_fwd(q, k, v, 0.125, window=band[0], sinks=band[1])
    torch.cuda.synchronize()
    assert _fronted(capfd.readouterr().err) == [want]


@pytest.mark.parametrize("size", SIZES, ids=_ids)
@pytest.mark.parametrize("band", BANDS, ids=_ids)
def test_values_and_gradients(size, band):
    q, k, v, do = _inputs(BF16, *size)
    for kind in ("whole", "padded", "newest", "anywhere"):
        _check_all(q, k, v, do, 0.125, window=band[0], sinks=band[1], **_ragged(kind, size[0], size[3], size[4]))


@pytest.mark.parametrize("layout", ["bhnd", "shared", "wide"])
@pytest.mark.parametrize("scale", [0.125, -0.3, 0.0])
def test_layouts_and_scales(layout, scale):
    size = (2, 4, 2, 400, 500)
    q, k, v, do = _inputs(BF16, *size, layout=layout, seed=3)
    _check_all(q, k, v, do, scale, window=128, sinks=5, **_ragged("newest", *size[:1], *size[3:]))


def test_heads_that_are_broadcast():
    q, k, v, do = _inputs(BF16, 2, 1, 1, 600, 600, seed=4)
    _check_all(q.expand(2, 4, 600, 64), k, v, do.expand(2, 4, 600, 64), 0.125, window=128, sinks=4)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("Nq", [300, 700])
def test_what_places_that_nobody_attends_hold_reaches_no_result(bad, Nq):
    size = (4, 4, 2, Nq, 700)
    q, k, v, do = _inputs(BF16, *size, layout="bhnd", seed=7)
    how = {"window": 128, "sinks": 4, "kv_len": _int32(333, 700, 0, 130), "q_start": _int32(333 - Nq + 2, 0, 0, 400)}
    seen = _seen(q, k, how)
    clean = _run(q, k, v, do, 0.125, **how)
    want = window(q, k, v, 0.125, seen, do, clean["O"])
    keys, queries = ~seen.any(1)[:, None, :, None], ~seen.any(2)[:, None, :, None]
    dirty = _run(q.masked_fill(queries, bad), k.masked_fill(keys, bad), v.masked_fill(keys, bad), do.masked_fill(queries, bad),
                 0.125, **how)
    for name in clean:
        check(name, clean[name], want[name])
        assert torch.equal(clean[name], dirty[name]), name


def test_captured_and_replayed_on_new_inputs():
    q, k, v, do = _inputs(BF16, 2, 4, 2, 600, 600, seed=9)
    how = {"window": 128, "sinks": 4, "kv_len": _int32(600, 411)}
    api.window_fwd(q, k, v, 0.125, **how)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = api.window_fwd(q, k, v, 0.125, **how)
    for seed in (10, 11):
        for t, new in zip((q, k, v), _inputs(BF16, 2, 4, 2, 600, 600, seed=seed)):
            t.copy_(new)
        how["kv_len"].copy_(_int32(500 + seed, 300))
        g.replay()
        want = api.window_fwd(q, k, v, 0.125, **how)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_more_units_than_the_gpu_holds():
    q, k, v, do = _inputs(BF16, 9, 12, 4, 1000, 1000, seed=12)
    _check_all(q, k, v, do, 0.125, window=128, sinks=4, **_ragged("padded", 9, 1000, 1000))


@pytest.mark.parametrize("dtype", [torch.float32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 4, 2, 300, 3), (3, 2, 2, 700, 129), (1, 6, 2, 65, 64), (2, 2, 1, 257, 33)], ids=_ids)
@pytest.mark.parametrize("band", [(None, 0), (2, 1), (20, 3), (32, 32)], ids=_ids)
def test_more_queries_than_keys(dtype, size, band):
    # most queries are outside their sequence, before it or behind it
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(dtype, *size, seed=13)
    for start in (0, -Nq + Nk, -Nq // 2, Nk - 1):
        got = _check_all(q, k, v, do, 0.125, window=band[0], sinks=band[1], q_start=_int32(*[start] * B))
        out = torch.arange(Nq, device="cuda") + start
        out = (out < 0) | (out >= Nk)
        assert bool((got["O"][:, :, out] == 0).all()) and bool((got["dQ"][:, :, out] == 0).all())
        assert bool((got["LSE"][:, :, out] == -math.inf).all())


@pytest.mark.parametrize("size", [(8, 6, 2, 640, 640), (3, 4, 4, 400, 400)], ids=_ids)
def test_gradients_of_padding_overwrite_what_was_there(size):
    # dQ of queries outside their sequence is cleared whatever its memory held, at its rows alone
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(BF16, *size, seed=14)
    how = {"window": 100, "sinks": 2, "kv_len": _int32(*[max(0, Nk - 97 * b) for b in range(B)])}
    o, lse = api.window_fwd(q, k, v, 0.125, **how)
    wide = torch.full((B, Nq, Hq, 72), math.nan, dtype=BF16, device="cuda")
    dq = wide[..., :64].transpose(1, 2)
    want = api.window_bwd(q, k, v, o, lse, do, 0.125, **how)
    got = api.window_bwd(q, k, v, o, lse, do, 0.125, **how, dQ=dq)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    out = torch.arange(Nq, device="cuda") >= how["kv_len"][:, None]
    assert bool((dq.transpose(1, 2)[out] == 0).all()) and bool(wide[..., 64:].isnan().all())
