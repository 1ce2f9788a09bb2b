"""The attention over a window with sinks on the GPU: values and gradients against
the definition in 64 bits (tests/window_ref.py, elementwise bounds from counted
roundings), over head layouts, windows, sinks, lengths, starts, strides and
scales; differences of the forward pass; streams, graphs and repeated calls."""
import math
import threading

import pytest
import torch

from test_cross_gpu import _inputs, _rand
from window_ref import check, seen_of, window
from sparse_head_self_gb300 import api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def _ids(s):
    return "x".join(map(str, s))


def _run(q, k, v, do, scale, **how):
    o, lse = api.window_fwd(q, k, v, scale, **how)
    dq, dk, dv = api.window_bwd(q, k, v, o, lse, do, scale, **how)
    torch.cuda.synchronize()
    return {"O": o, "LSE": lse, "dQ": dq, "dK": dk, "dV": dv}


def _seen(q, k, how):
    return seen_of(q.shape[0], q.shape[2], k.shape[2], how.get("window"), how.get("sinks", 0), how.get("q_start"),
                   how.get("kv_len"), q.device)


def _check_all(q, k, v, do, scale, **how):
    got = _run(q, k, v, do, scale, **how)
    want = window(q, k, v, scale, _seen(q, k, how), do, got["O"])
    for name in got:
        check(name, got[name], want[name])
    return got


def _int32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _ragged(kind, B, Nq, Nk, seed=1):
    """q_start and kv_len of sequences of several lengths: padded behind, or a part of the newest tokens."""
    if kind == "whole":
        return {}
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = torch.randint(0, Nk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = Nk if B == 1 else 0
    if kind == "padded":
        return {"kv_len": n}
    if kind == "newest":
        return {"q_start": n - Nq, "kv_len": n}
    # anywhere: before, across and behind the keys
    return {"q_start": torch.randint(-Nq, Nk + 1, (B,), generator=g, device="cuda", dtype=torch.int32), "kv_len": n}


SIZES = [  # B, Hq, Hkv, Nq, Nk
    (1, 1, 1, 1, 1), (2, 4, 2, 1, 7), (4, 3, 3, 2, 2), (3, 2, 2, 64, 64), (2, 3, 3, 65, 65), (2, 4, 1, 127, 129),
    (2, 2, 2, 128, 128), (1, 1, 1, 129, 257), (2, 6, 2, 197, 197), (1, 3, 1, 33, 1000), (2, 16, 4, 1, 1569),
    (2, 8, 1, 3, 400), (3, 4, 4, 16, 513), (2, 3, 1, 300, 300), (2, 4, 2, 260, 700), (1, 5, 5, 700, 700), (5, 1, 1, 9, 130),
]
BANDS = [(None, 0), (1, 0), (5, 2), (64, 1), (100, 70), (128, 4), (200, 130), (400, 0)]


@TYPES
@pytest.mark.parametrize("size", SIZES, ids=_ids)
@pytest.mark.parametrize("band", BANDS, ids=_ids)
def test_values_and_gradients(dtype, size, band):
    q, k, v, do = _inputs(dtype, *size)
    for kind in ("whole", "padded", "newest", "anywhere"):
        _check_all(q, k, v, do, 0.125, window=band[0], sinks=band[1], **_ragged(kind, size[0], size[3], size[4]))


@TYPES
@pytest.mark.parametrize("layout", ["bhnd", "shared", "wide"])
@pytest.mark.parametrize("size", [(3, 4, 2, 70, 150), (2, 4, 4, 1, 300), (2, 2, 1, 200, 210)], ids=_ids)
def test_layouts(dtype, layout, size):
    q, k, v, do = _inputs(dtype, *size, layout=layout)
    _check_all(q, k, v, do, 0.125, window=60, sinks=3, **_ragged("newest", size[0], size[3], size[4]))


@TYPES
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
@pytest.mark.parametrize("size", [(2, 2, 2, 70, 200), (2, 4, 1, 1, 200), (1, 4, 2, 300, 300)], ids=_ids)
def test_scales(dtype, scale, size):
    q, k, v, do = _inputs(dtype, *size, seed=3)
    _check_all(q, k, v, do, scale, window=90, sinks=5)


@TYPES
@pytest.mark.parametrize("Nq", [1, 6, 100, 600])
def test_large_scores_in_growing_order(dtype, Nq):
    q, k, v, do = _inputs(dtype, 1, 2, 2, Nq, 600, seed=5)
    q = (q.abs() * 2).to(dtype)
    k = (k.abs() * (torch.arange(600, device="cuda")[:, None] / 150.0)).to(dtype)
    _check_all(q, k, v, do, 0.125, window=350, sinks=4)


@TYPES
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("size", [(3, 4, 2, 70, 300), (3, 4, 2, 1, 300), (3, 4, 2, 300, 300), (3, 2, 2, 5, 300)], ids=_ids)
@pytest.mark.parametrize("band", [(40, 3), (130, 0), (None, 0)], ids=_ids)
def test_what_places_that_nobody_attends_hold_reaches_no_result(dtype, bad, size, band):
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(dtype, *size, layout="bhnd", seed=7)
    n = _int32(137, 300, 0)
    how = {"window": band[0], "sinks": band[1], "kv_len": n}
    if Nq < Nk:
        how["q_start"] = n - Nq + _int32(2, -20, 0)
    seen = _seen(q, k, how)
    clean = _run(q, k, v, do, 0.125, **how)
    want = window(q, k, v, 0.125, seen, do, clean["O"])
    keys, queries = ~seen.any(1)[:, None, :, None], ~seen.any(2)[:, None, :, None]
    k2, v2 = k.masked_fill(keys, bad), v.masked_fill(keys, bad)
    q2, do2 = q.masked_fill(queries, bad), do.masked_fill(queries, bad)
    dirty = _run(q2, k2, v2, do2, 0.125, **how)
    for name in clean:
        check(name, clean[name], want[name])
        assert torch.equal(clean[name], dirty[name]), name
    for name, dead in (("dK", keys), ("dV", keys), ("O", queries), ("dQ", queries)):
        assert bool((dirty[name].masked_select(dead) == 0).all()), name
    assert bool((dirty["LSE"].masked_select(queries[..., 0]) == -math.inf).all())


@TYPES
@pytest.mark.parametrize("Nq", [1, 40, 300])
def test_lengths_and_starts_outside_their_range(dtype, Nq):
    q, k, v, do = _inputs(dtype, 5, 2, 2, Nq, 300)
    far = 2 ** 31 - 1
    got = _check_all(q, k, v, do, 0.125, window=50, sinks=2, q_start=_int32(-far - 1, far, 0, -Nq + 1, 299),
                     kv_len=_int32(far, far, -5, far, 300))
    assert bool((got["O"][:3] == 0).all()) and bool((got["LSE"][:3] == -math.inf).all())
    assert bool((got["dK"][:3] == 0).all())


@pytest.mark.parametrize("sizes", [(2 ** 31 - 1, 0), (300, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (10 ** 12, 10 ** 12)], ids=_ids)
def test_windows_and_sinks_beyond_the_keys_are_all_of_them(sizes):
    q, k, v, do = _inputs(BF16, 2, 4, 2, 300, 300)
    got, want = _run(q, k, v, do, 0.125, window=sizes[0], sinks=sizes[1]), _run(q, k, v, do, 0.125)
    for name in got:
        assert torch.equal(got[name], want[name]), name


@TYPES
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 16385), (1, 2, 1, 40, 16385), (1, 4, 1, 2000, 9000), (1, 2, 2, 4500, 4500)], ids=_ids)
@pytest.mark.parametrize("band", [(1000, 4), (None, 0), (130, 300)], ids=_ids)
def test_long_sequences(dtype, size, band):
    q, k, v, do = _inputs(dtype, *size, seed=11)
    _check_all(q, k, v, do, 0.125, window=band[0], sinks=band[1])


@TYPES
@pytest.mark.parametrize("Nq", [1, 70])
def test_offsets_past_32_bits(dtype, Nq):
    # rows 128 K elements apart: the last ones start 2.6e9 elements behind the first
    Nk, step = 20000, 1 << 17
    store = torch.empty(Nk * step, dtype=dtype, device="cuda")
    k = torch.as_strided(store, (1, 1, Nk, 64), (Nk * step, Nk * step, step, 1))
    v = torch.as_strided(store, (1, 1, Nk, 64), (Nk * step, Nk * step, step, 1), 64)
    q, k0, v0, do = _inputs(dtype, 1, 1, 1, Nq, Nk, layout="bhnd")
    k.copy_(k0)
    v.copy_(v0)
    how = {"window": 700, "sinks": 4}
    got = _run(q, k, v, do, 0.125, **how)
    want = window(q, k0, v0, 0.125, _seen(q, k, how), do, got["O"])
    for name in got:
        check(name, got[name], want[name])
    dk, dv = torch.empty_like(k0), torch.empty_like(v0)
    dk_far = torch.as_strided(store, (1, 1, Nk, 64), (Nk * step, Nk * step, step, 1), 128)
    o, lse = api.window_fwd(q, k, v, 0.125, **how)
    api.window_bwd(q, k, v, o, lse, do, 0.125, dK=dk_far, dV=dv, **how)
    api.window_bwd(q, k, v, o, lse, do, 0.125, dK=dk, dV=dv, **how)
    assert torch.equal(dk_far, dk)


@TYPES
@pytest.mark.parametrize("size", [(2, 4, 2, 100, 200), (2, 4, 2, 1, 200), (1, 2, 2, 129, 130)], ids=_ids)
def test_only_the_results_rows_are_written(dtype, size):
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(dtype, *size)
    how = {"window": 77, "sinks": 2}

    def inside(H, N):   # a tensor within a larger one full of a mark
        big = torch.full((B, N + 5, H + 2, 80), 77.0, dtype=dtype, device="cuda")
        return big, big[:, 2:2 + N, 1:1 + H, 8:72].transpose(1, 2)

    bigs = {name: inside(H, N) for name, H, N in (("O", Hq, Nq), ("dQ", Hq, Nq), ("dK", Hkv, Nk), ("dV", Hkv, Nk))}
    o, lse = api.window_fwd(q, k, v, 0.125, O=bigs["O"][1], **how)
    api.window_bwd(q, k, v, o, lse, do, 0.125, dQ=bigs["dQ"][1], dK=bigs["dK"][1], dV=bigs["dV"][1], **how)
    ref = _run(q, k, v, do, 0.125, **how)
    for name, (big, view) in bigs.items():
        assert torch.equal(view, ref[name]), name
        view.fill_(77.0)
        assert bool((big == 77.0).all()), name


@pytest.mark.parametrize("size", [(2, 4, 2, 50, 50), (1, 2, 2, 3, 40)], ids=_ids)
def test_gradients_against_differences(size):
    # central differences of <O, dO> along a random direction: the kernels' against the
    # definition's at the same step (whose truncation is thereby known), each forward
    # value within its bound
    how = {"window": 20, "sinks": 3}
    q, k, v, do = _inputs(F32, *size, seed=13)
    seen = _seen(q, k, how)
    got = _run(q, k, v, do, 0.125, **how)
    step = 2.0 ** -6
    g = torch.Generator(device="cuda").manual_seed(17)
    for name, x in (("dQ", 0), ("dK", 1), ("dV", 2)):
        xs = [q, k, v]
        d = torch.randn(xs[x].shape, generator=g, device="cuda")
        vals, refs, slack = [], [], 0.0
        for sign in (1, -1):
            ys = list(xs)
            ys[x] = xs[x] + sign * step * d
            o, _ = api.window_fwd(*ys, 0.125, **how)
            ref, bound = window(*ys, 0.125, seen)["O"]
            vals.append(float((o.double() * do.double()).sum()))
            refs.append(float((ref * do.double()).sum()))
            slack += float((bound * do.double().abs()).sum())
        want, bound = window(q, k, v, 0.125, seen, do, got["O"])[name]
        # the step itself is rounded to 32 bits: half a unit of |x| + step |d| each way
        moved = (xs[x].abs().double() + step * d.abs().double()) * 2.0 ** -24 / step
        slack = slack / (2 * step) + float((want.abs() * moved).sum()) * 1.1
        kernel = (vals[0] - vals[1]) / (2 * step)
        exact = (refs[0] - refs[1]) / (2 * step)
        along = float((got[name].double() * d.double()).sum())
        truth = float((want * d.double()).sum())
        assert abs(kernel - exact) <= slack, name
        assert abs(along - truth) <= float((bound * d.double().abs()).sum()), name
        assert abs(kernel - along) <= slack + abs(exact - truth) + float((bound * d.double().abs()).sum()), name


@TYPES
@pytest.mark.parametrize("size", [(2, 4, 2, 150, 300), (2, 4, 2, 1, 900), (1, 4, 1, 600, 600)], ids=_ids)
def test_the_same_result_on_every_call(dtype, size):
    q, k, v, do = _inputs(dtype, *size)
    how = {"window": 200, "sinks": 4, **_ragged("newest", size[0], size[3], size[4])}
    first = _run(q, k, v, do, 0.125, **how)
    for _ in range(3):
        again = _run(q, k, v, do, 0.125, **how)
        for name in first:
            assert torch.equal(first[name], again[name]), name


@TYPES
@pytest.mark.parametrize("Nq", [1, 130])
def test_streams_and_two_calls_at_once(dtype, Nq):
    how = {"window": 300, "sinks": 4}
    sets = [_inputs(dtype, 2, 4, 2, Nq, 700, seed=s) for s in (1, 2)]
    want = [_run(*s, 0.125, **how) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(4):
        for i, (s, (q, k, v, do)) in enumerate(zip(streams, sets)):
            o, lse = api.window_fwd(q, k, v, 0.125, stream=s, **how)
            got[i].append((o, lse) + api.window_bwd(q, k, v, o, lse, do, 0.125, stream=s, **how))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for r in g:
            for name, t in zip(("O", "LSE", "dQ", "dK", "dV"), r):
                assert torch.equal(w[name], t), name


@TYPES
@pytest.mark.parametrize("Nq", [1, 70])
def test_captured_and_replayed_on_new_inputs(dtype, Nq):
    q, k, v, do = (t.contiguous() for t in _inputs(dtype, 2, 4, 2, Nq, 333, layout="bhnd"))
    n, start = _int32(333, 100), _int32(333 - Nq, 100 - Nq)
    how = {"window": 120, "sinks": 2, "q_start": start, "kv_len": n}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _run(q, k, v, do, 0.125, **how)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = api.window_fwd(q, k, v, 0.125, **how)
        grads = api.window_bwd(q, k, v, o, lse, do, 0.125, **how)
    for seed in (21, 22):
        for t, new in zip((q, k, v, do), _inputs(dtype, 2, 4, 2, Nq, 333, layout="bhnd", seed=seed)):
            t.copy_(new)
        n.copy_(_int32(seed, 200 + seed))       # lengths and starts are read on the device
        start.copy_(n - Nq)
        graph.replay()
        torch.cuda.synchronize()
        want = _run(q, k, v, do, 0.125, **how)
        for name, t in zip(("O", "LSE", "dQ", "dK", "dV"), (o, lse) + tuple(grads)):
            assert torch.equal(want[name], t), name


@TYPES
@pytest.mark.parametrize("Nq", [1, 70])
def test_from_threads_that_made_no_other_call(dtype, Nq):
    q, k, v, do = _inputs(dtype, 2, 4, 2, Nq, 90)
    want = _run(q, k, v, do, 0.125, window=30)
    got = {}

    def fwd():
        got["O"], got["LSE"] = api.window_fwd(q, k, v, 0.125, window=30)

    def bwd():
        got["dQ"], got["dK"], got["dV"] = api.window_bwd(q, k, v, want["O"], want["LSE"], do, 0.125, window=30)

    for f in (fwd, bwd):
        t = threading.Thread(target=f)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert set(got) == set(want)
    for name in want:
        assert torch.equal(want[name], got[name]), name


@TYPES
def test_autograd_with_odd_layouts_and_broadcast_gradients(dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = _rand(g, 2, 90, 4 * 64 + 2 * 2 * 64 + 1, dtype=dtype).requires_grad_()      # rows off 16 bytes: copied
    q = qkv[..., 1:257].view(2, 90, 4, 64).transpose(1, 2)
    k, v = (qkv[..., a:a + 128].view(2, 90, 2, 64).transpose(1, 2) for a in (257, 385))
    w = _rand(g, 2, 4, 64, dtype=dtype)
    n = _int32(90, 41)
    o = api.window_attention(q, k, v, window=30, sinks=2, kv_len=n)
    (o.sum(2) * w).sum().backward()           # rows of dO with a stride of 0
    do = w[:, :, None].expand_as(o)
    want = window(q.detach(), k.detach(), v.detach(), 0.125, seen_of(2, 90, 90, 30, 2, None, n), do, o.detach())
    check("O", o.detach(), want["O"])
    check("dQ", qkv.grad[..., 1:257].view(2, 90, 4, 64).transpose(1, 2), want["dQ"])
    for a, name in ((257, "dK"), (385, "dV")):
        check(name, qkv.grad[..., a:a + 128].view(2, 90, 2, 64).transpose(1, 2), want[name])
    assert bool((qkv.grad[..., 0] == 0).all())


@TYPES
@pytest.mark.parametrize("Nq", [1, 50, 150])
def test_heads_that_are_broadcast(dtype, Nq):
    # one row of queries (and of dO) for all heads, one key head for all
    g = torch.Generator(device="cuda").manual_seed(31)
    q, do = (_rand(g, 2, 1, Nq, 64, dtype=dtype).expand(-1, 6, -1, -1) for _ in range(2))
    k, v = (_rand(g, 2, 1, 160, 64, dtype=dtype).expand(-1, 3, -1, -1) for _ in range(2))
    _check_all(q, k, v, do, 0.125, window=70, sinks=1)


@TYPES
@pytest.mark.parametrize("size", [(40, 2, 2, 150, 260), (6, 24, 2, 40, 700), (3, 12, 12, 1, 5000), (50, 12, 4, 6, 90),
                                  (2, 32, 2, 1, 300), (110, 6, 6, 20, 200), (60, 8, 8, 130, 300), (9, 4, 2, 1000, 1000)], ids=_ids)
@pytest.mark.parametrize("band", [(150, 4), (None, 0)], ids=_ids)
def test_more_units_than_the_gpu_holds(dtype, size, band):
    q, k, v, do = _inputs(dtype, *size, seed=37)
    how = _ragged("newest" if size[3] < size[4] else "padded", size[0], size[3], size[4], seed=3)
    how["kv_len"][size[0] // 3:size[0] // 2] = 0       # runs of units without keys
    _check_all(q, k, v, do, 0.125, window=band[0], sinks=band[1], **how)


@TYPES
@pytest.mark.parametrize("size", [(2, 6, 2, 50, 150), (1, 9, 3, 33, 300), (2, 10, 2, 1, 70)], ids=_ids)
@pytest.mark.parametrize("bad", [math.nan, 1e6])
def test_other_groups_queries_reach_no_gradient(dtype, size, bad):
    q, k, v, do = _inputs(dtype, *size, layout="bhnd", seed=41)
    G = size[1] // size[2]
    want = _run(q, k, v, do, 0.125, window=60, sinks=2)
    q, do = q.clone(), do.clone()
    q[:, G:] = bad
    do[:, G:] = bad
    got = _run(q, k, v, do, 0.125, window=60, sinks=2)
    for name, n in (("O", G), ("LSE", G), ("dQ", G), ("dK", 1), ("dV", 1)):
        assert torch.equal(got[name][:, :n], want[name][:, :n]), name


@TYPES
@pytest.mark.parametrize("size", [(2, 4, 2, 300, 300), (2, 4, 2, 40, 300), (2, 4, 2, 2, 300)], ids=_ids)
def test_nan_in_an_attended_place_stays_near_its_queries(dtype, size):
    # the queries that attend the key have it; those more than 255 rows away, other heads and sequences do not
    q, k, v, do = _inputs(dtype, *size, layout="bhnd", seed=43)
    want = _run(q, k, v, do, 0.125, window=20)
    seen = seen_of(*size[:1], *size[3:], 20)[0, :, 295]
    k[0, 0, 295, 3] = math.nan
    got = _run(q, k, v, do, 0.125, window=20)
    assert bool(seen.any())
    for name in ("O", "LSE", "dQ"):
        assert bool(got[name][0, :2, seen].isnan().all()), name
        assert torch.equal(got[name][0, 2:], want[name][0, 2:]) and torch.equal(got[name][1], want[name][1]), name
        far = torch.arange(size[3], device="cuda") + 255 < seen.nonzero()[0]
        assert torch.equal(got[name][0, :2, far], want[name][0, :2, far]), name


def test_a_long_walk_next_to_short_ones():
    # the first keys' tile is attended by all queries of four heads, the others by a window's
    q, k, v, do = _inputs(BF16, 2, 8, 2, 5000, 5000, seed=61)
    got = _run(q, k, v, do, 0.125, window=100, sinks=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    for b, hk in ((0, 0), (1, 1)):
        hq = slice(4 * hk, 4 * hk + 4)
        at = [t[b:b + 1, hq] for t in (q, do, got["O"], got["dQ"], got["LSE"])]
        kk, vv = k[b:b + 1, hk:hk + 1], v[b:b + 1, hk:hk + 1]
        want = window(at[0], kk, vv, 0.125, seen_of(1, 5000, 5000, 100, 4), at[1], at[2])
        for name, t in (("O", at[2]), ("LSE", at[4]), ("dQ", at[3]), ("dK", got["dK"][b:b + 1, hk:hk + 1]),
                        ("dV", got["dV"][b:b + 1, hk:hk + 1])):
            check(name, t, want[name])


@pytest.mark.parametrize("size,band", [((8, 4, 4, 60, 60), (3, 0)), ((8, 4, 4, 60, 60), (8, 1)), ((8, 4, 2, 5, 300), (4, 2)),
                                       ((8, 4, 2, 700, 700), (6, 2)), ((8, 4, 2, 40, 500), (40, 4)), ((200, 4, 2, 7, 7), (None, 0)),
                                       ((60, 4, 4, 20, 20), (None, 0)), ((2, 4, 2, 1000, 1000), (50, 14)), ((20, 4, 2, 33, 64), (64, 0))],
                         ids=_ids)
def test_gradients_of_few_keys_have_two_roundings(size, band):
    # dS and the result are each rounded once to 16 bits: at most 2^-8 of the value, uniform below
    # that, so 2^-8 / sqrt(3) in the mean square; two independent ones are sqrt(2) of it
    q, k, v, do = _inputs(BF16, *size, layout="bhnd", seed=53)
    how = {"window": band[0], "sinks": band[1]}
    got = _check_all(q, k, v, do, 0.125, **how)
    G = size[1] // size[2]
    x, y, z, w = q.double(), *(t.double().repeat_interleave(G, 1) for t in (k, v)), do.double()
    s = (0.125 * x @ y.transpose(-1, -2)).masked_fill(~_seen(q, k, how)[:, None], -math.inf)
    p, dp = s.softmax(-1), w @ z.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dk = (0.125 * ds.transpose(-1, -2) @ x).view(size[0], size[2], G, size[4], 64).sum(2)
    for name, exact in (("dQ", 0.125 * ds @ y), ("dK", dk)):
        err = float((got[name].double() - exact).norm() / exact.norm())
        assert err <= math.sqrt(2 / 3) * 2.0 ** -8, (name, err)


def test_gradients_of_gradients_are_refused():
    q, k, v, _ = (t.detach().clone().requires_grad_() for t in _inputs(F32, 1, 2, 2, 5, 9))
    dq, = torch.autograd.grad(api.window_attention(q, k, v).square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dq.sum().backward()


def test_gpu_refusals():
    q, k, v, do = _inputs(BF16, 2, 4, 2, 5, 9)
    with pytest.raises(ValueError, match="q_start"):
        api.window_fwd(q, k, v, 0.125, q_start=torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="kv_len"):
        api.window_fwd(q, k, v, 0.125, kv_len=torch.ones(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(api.FibattError, match="window"):
        api.window_fwd(q, k, v, 0.125, window=0)
    with pytest.raises(api.FibattError, match="sinks"):
        api.window_fwd(q, k, v, 0.125, window=4, sinks=-1)
    with pytest.raises(TypeError):
        api.window_fwd(q, k, v, 0.125, window=4.5)
    with pytest.raises(api.FibattError, match="q_start"):
        api.window_fwd(q, k[:, :, :4], v[:, :, :4], 0.125)
    o, lse = api.window_fwd(q, k, v, 0.125)
    with pytest.raises(api.FibattError, match="workspace"):
        api.window_bwd(q, k, v, o, lse, do, 0.125, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
