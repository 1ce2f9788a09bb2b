"""The cross attention on the GPU: values and gradients against the definition
in 64 bits (tests/cross_ref.py, elementwise bounds from counted roundings),
over head layouts, lengths, masks, strides and scales; differences of the
forward pass; streams, graphs and repeated calls."""
import math
import threading

import pytest
import torch

from cross_ref import check, cross
from sparse_head_self_gb300 import api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _rand(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _inputs(dtype, B, Hq, Hkv, Nq, Nk, layout="bnhd", seed=0, grow=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "bhnd":
        q, do = _rand(g, B, Hq, Nq, 64, dtype=dtype), _rand(g, B, Hq, Nq, 64, dtype=dtype)
        k, v = _rand(g, B, Hkv, Nk, 64, dtype=dtype), _rand(g, B, Hkv, Nk, 64, dtype=dtype)
    elif layout == "shared":      # the same states for every sequence: a stride of 0
        q, do = _rand(g, B, Hq, Nq, 64, dtype=dtype), _rand(g, B, Hq, Nq, 64, dtype=dtype)
        k, v = (_rand(g, 1, Hkv, Nk, 64, dtype=dtype).expand(B, -1, -1, -1) for _ in range(2))
    elif layout == "wide":        # rows far apart, an odd number of 16-byte steps
        q, do = (_rand(g, B, Nq, Hq, 72, dtype=dtype)[..., 8:].transpose(1, 2) for _ in range(2))
        k, v = (_rand(g, B, Hkv, Nk, 104, dtype=dtype)[..., 16:80] for _ in range(2))
    else:                          # as projections leave them
        q, do = (_rand(g, B, Nq, Hq, 64, dtype=dtype).transpose(1, 2) for _ in range(2))
        kv = _rand(g, B, Nk, 2, Hkv, 64, dtype=dtype)
        k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    return q * grow, k, v, do


def _masks(kind, B, Nk, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = m = None
    if kind in ("len", "both"):
        n = torch.randint(0, Nk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = Nk if B == 1 else 0      # a sequence without keys next to others
    if kind in ("mask", "both"):
        m = torch.rand(B, Nk, generator=g, device="cuda") < 0.6
        if B > 1:
            m[B - 1] = False
        if B > 2:
            m[1, :-1] = False           # one key: the last
            m[1, -1] = True
    return n, m


def _run(q, k, v, do, scale, n=None, m=None):
    o, lse = api.cross_fwd(q, k, v, scale, n, m)
    dq, dk, dv = api.cross_bwd(q, k, v, o, lse, do, scale, n, m)
    torch.cuda.synchronize()
    return {"O": o, "LSE": lse, "dQ": dq, "dK": dk, "dV": dv}


def _check_all(q, k, v, do, scale, n=None, m=None):
    got = _run(q, k, v, do, scale, n, m)
    want = cross(q, k, v, scale, n, m, do, got["O"])
    for name in got:
        check(name, got[name], want[name])
    return got


SIZES = [  # B, Hq, Hkv, Nq, Nk
    (1, 1, 1, 1, 1), (2, 4, 2, 1, 7), (1, 2, 1, 5, 1), (4, 3, 3, 2, 2), (2, 3, 3, 64, 64), (3, 2, 2, 65, 63),
    (2, 4, 1, 127, 129), (1, 2, 2, 128, 128), (1, 1, 1, 129, 257), (2, 6, 2, 197, 197), (1, 3, 1, 33, 1000),
    (1, 2, 2, 300, 77), (3, 4, 4, 16, 513), (2, 16, 4, 1, 1569), (2, 8, 1, 3, 400), (1, 1, 1, 700, 31), (5, 1, 1, 9, 130),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("mask", ["none", "len", "mask", "both"])
def test_values_and_gradients(dtype, size, mask):
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(dtype, *size)
    _check_all(q, k, v, do, 0.125, *_masks(mask, B, Nk))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bhnd", "shared", "wide"])
@pytest.mark.parametrize("size", [(3, 4, 2, 70, 150), (2, 4, 4, 1, 300), (2, 2, 1, 200, 40)],
                         ids=lambda s: "x".join(map(str, s)))
def test_layouts(dtype, layout, size):
    q, k, v, do = _inputs(dtype, *size, layout=layout)
    _check_all(q, k, v, do, 0.125, *_masks("both", size[0], size[4]))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
@pytest.mark.parametrize("size", [(2, 2, 2, 70, 200), (2, 4, 1, 1, 200)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("mask", ["none", "both"])
def test_scales(dtype, scale, size, mask):
    q, k, v, do = _inputs(dtype, *size, seed=3)
    _check_all(q, k, v, do, scale, *_masks(mask, size[0], size[4]))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 6, 100])
def test_large_scores_in_growing_order(dtype, Nq):
    # each tile's maximum is far above the last one's: every running maximum moves
    q, k, v, do = _inputs(dtype, 1, 2, 2, Nq, 600, seed=5)
    q = (q.abs() * 2).to(dtype)
    k = (k.abs() * (torch.arange(600, device="cuda")[:, None] / 150.0)).to(dtype)
    _check_all(q, k, v, do, 0.125)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("size", [(2, 4, 2, 70, 300), (2, 4, 2, 1, 300)], ids=lambda s: "x".join(map(str, s)))
def test_what_masked_places_hold_reaches_no_result(dtype, bad, size):
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(dtype, *size, layout="bhnd", seed=7)
    n = torch.tensor([137, 300], dtype=torch.int32, device="cuda")
    m = torch.rand(B, Nk, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) < 0.7
    m[1, 128:256] = False       # a whole tile masked between two that are not
    keep = (torch.arange(Nk, device="cuda")[None] < n[:, None]) & m
    dead = ~keep[:, None, :, None]
    clean = _run(q, k, v, do, 0.125, n, m)
    k2, v2 = k.masked_fill(dead, bad), v.masked_fill(dead, bad)
    dirty = _run(q, k2, v2, do, 0.125, n, m)
    want = cross(q, k, v, 0.125, n, m, do, clean["O"])
    for name in clean:
        check(name, clean[name], want[name])
        assert torch.equal(clean[name], dirty[name]), name
    for name in ("dK", "dV"):
        assert bool((dirty[name].masked_select(dead) == 0).all()), name


def test_lengths_outside_their_range_are_clamped():
    q, k, v, do = _inputs(BF16, 3, 2, 2, 40, 90)
    n = torch.tensor([-5, 2**31 - 1, 90], dtype=torch.int32, device="cuda")
    got = _check_all(q, k, v, do, 0.125, n)
    assert bool((got["O"][0] == 0).all()) and bool((got["LSE"][0] == -math.inf).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 16385), (1, 2, 1, 40, 16385), (1, 1, 1, 16385, 70), (2, 4, 4, 300, 4100)],
                         ids=lambda s: "x".join(map(str, s)))
def test_long_sequences(dtype, size):
    q, k, v, do = _inputs(dtype, *size, seed=11)
    n = torch.full((size[0],), size[4] - 3, dtype=torch.int32, device="cuda")
    _check_all(q, k, v, do, 0.125, n)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
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
    got = _run(q, k, v, do, 0.125)
    want = cross(q, k0, v0, 0.125, None, None, do, got["O"])
    for name in got:
        check(name, got[name], want[name])
    # gradients written that far apart, too
    dk, dv = torch.empty_like(k0), torch.empty_like(v0)
    dk_far = torch.as_strided(store, (1, 1, Nk, 64), (Nk * step, Nk * step, step, 1), 128)
    o, lse = api.cross_fwd(q, k, v, 0.125)
    api.cross_bwd(q, k, v, o, lse, do, 0.125, dK=dk_far, dV=dv)
    api.cross_bwd(q, k, v, o, lse, do, 0.125, dK=dk, dV=dv)
    assert torch.equal(dk_far, dk)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 4, 2, 100, 200), (2, 4, 2, 1, 200), (1, 2, 2, 129, 65)],
                         ids=lambda s: "x".join(map(str, s)))
def test_only_the_results_rows_are_written(dtype, size):
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(dtype, *size)

    def inside(H, N):   # a tensor within a larger one full of a mark
        big = torch.full((B, N + 5, H + 2, 80), 77.0, dtype=dtype, device="cuda")
        return big, big[:, 2:2 + N, 1:1 + H, 8:72].transpose(1, 2)

    bigs = {}
    for name, H, N in (("O", Hq, Nq), ("dQ", Hq, Nq), ("dK", Hkv, Nk), ("dV", Hkv, Nk)):
        bigs[name] = inside(H, N)
    o, lse = api.cross_fwd(q, k, v, 0.125, O=bigs["O"][1])
    api.cross_bwd(q, k, v, o, lse, do, 0.125, dQ=bigs["dQ"][1], dK=bigs["dK"][1], dV=bigs["dV"][1])
    ref = _run(q, k, v, do, 0.125)
    for name, (big, view) in bigs.items():
        assert torch.equal(view, ref[name]), name
        view.fill_(77.0)
        assert bool((big == 77.0).all()), name


@pytest.mark.parametrize("size", [(2, 4, 2, 20, 50), (1, 2, 2, 1, 40)], ids=lambda s: "x".join(map(str, s)))
def test_gradients_against_differences(size):
    # central differences of <O, dO> along a random direction: the kernels' against
    # the definition's at the same step (whose truncation is thereby known), each
    # forward value within its bound
    q, k, v, do = _inputs(F32, *size, seed=13)
    got = _run(q, k, v, do, 0.125)
    step = 2.0 ** -6
    g = torch.Generator(device="cuda").manual_seed(17)
    for name, x in (("dQ", 0), ("dK", 1), ("dV", 2)):
        xs = [q, k, v]
        d = torch.randn(xs[x].shape, generator=g, device="cuda")
        vals, refs, slack = [], [], 0.0
        for sign in (1, -1):
            ys = list(xs)
            ys[x] = xs[x] + sign * step * d
            o, _ = api.cross_fwd(*ys, 0.125)
            ref, bound = cross(*ys, 0.125)["O"]
            vals.append(float((o.double() * do.double()).sum()))
            refs.append(float((ref * do.double()).sum()))
            slack += float((bound * do.double().abs()).sum())
        want, bound = cross(q, k, v, 0.125, None, None, do, got["O"])[name]
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


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 4, 2, 150, 300), (2, 4, 2, 1, 900), (1, 4, 1, 600, 40)],
                         ids=lambda s: "x".join(map(str, s)))
def test_the_same_result_on_every_call(dtype, size):
    q, k, v, do = _inputs(dtype, *size)
    n, m = _masks("both", size[0], size[4])
    first = _run(q, k, v, do, 0.125, n, m)
    for _ in range(3):
        again = _run(q, k, v, do, 0.125, n, m)
        for name in first:
            assert torch.equal(first[name], again[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 130])
def test_streams_and_two_calls_at_once(dtype, Nq):
    sets = [_inputs(dtype, 2, 4, 2, Nq, 700, seed=s) for s in (1, 2)]
    want = [_run(*s, 0.125) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(4):
        for i, (s, (q, k, v, do)) in enumerate(zip(streams, sets)):
            o, lse = api.cross_fwd(q, k, v, 0.125, stream=s)
            got[i].append((o, lse) + api.cross_bwd(q, k, v, o, lse, do, 0.125, stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for r in g:
            for name, t in zip(("O", "LSE", "dQ", "dK", "dV"), r):
                assert torch.equal(w[name], t), name


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 70])
def test_captured_and_replayed_on_new_inputs(dtype, Nq):
    q, k, v, do = (t.contiguous() for t in _inputs(dtype, 2, 4, 2, Nq, 333, layout="bhnd"))
    n = torch.tensor([333, 100], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _run(q, k, v, do, 0.125, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = api.cross_fwd(q, k, v, 0.125, n)
        grads = api.cross_bwd(q, k, v, o, lse, do, 0.125, n)
    for seed in (21, 22):
        for t, new in zip((q, k, v, do), _inputs(dtype, 2, 4, 2, Nq, 333, layout="bhnd", seed=seed)):
            t.copy_(new)
        n.copy_(torch.tensor([seed, 200 + seed], dtype=torch.int32, device="cuda"))   # lengths are read on the device
        graph.replay()
        torch.cuda.synchronize()
        want = _run(q, k, v, do, 0.125, n)
        for name, t in zip(("O", "LSE", "dQ", "dK", "dV"), (o, lse) + tuple(grads)):
            assert torch.equal(want[name], t), name


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 70])
def test_from_threads_that_made_no_other_call(dtype, Nq):
    # a fresh thread has no current context until something makes the device's current
    q, k, v, do = _inputs(dtype, 2, 4, 2, Nq, 90)
    want = _run(q, k, v, do, 0.125)
    got = {}

    def fwd():
        got["O"], got["LSE"] = api.cross_fwd(q, k, v, 0.125)

    def bwd():
        got["dQ"], got["dK"], got["dV"] = api.cross_bwd(q, k, v, want["O"], want["LSE"], do, 0.125)

    for f in (fwd, bwd):
        t = threading.Thread(target=f)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert set(got) == set(want)
    for name in want:
        assert torch.equal(want[name], got[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_autograd_with_shared_states_and_odd_layouts(dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    q = _rand(g, 3, 4, 30, 64, dtype=dtype).requires_grad_()
    kv = _rand(g, 1, 2, 50, 2 * 64 + 1, dtype=dtype).requires_grad_()    # rows off 16 bytes: copied
    k, v = kv[..., 1:65].expand(3, -1, -1, -1), kv[..., 65:].expand(3, -1, -1, -1)
    do = _rand(g, 3, 4, 30, 64, dtype=dtype)
    o = api.cross_attention(q, k, v)
    o.backward(do)
    want = cross(q.detach(), k.detach(), v.detach(), 0.125, None, None, do, o.detach())
    check("O", o.detach(), want["O"])
    check("dQ", q.grad, want["dQ"])
    # autograd adds the three sequences' gradients in the I/O type
    for at, name in ((slice(1, 65), "dK"), (slice(65, None), "dV")):
        value, bound = want[name]
        h = torch.finfo(dtype).eps / 2
        check(name, kv.grad[..., at], (value.sum(0, keepdim=True), bound.sum(0, keepdim=True) + 3 * h * (value.abs() + bound).sum(0, keepdim=True)))
    assert bool((kv.grad[..., 0] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 50, 150])
def test_heads_and_masks_that_are_broadcast(dtype, Nq):
    # one row of queries (and of dO) for all heads, one key head for all, one mask for all sequences
    g = torch.Generator(device="cuda").manual_seed(31)
    q, do = (_rand(g, 2, 1, Nq, 64, dtype=dtype).expand(-1, 6, -1, -1) for _ in range(2))
    k, v = (_rand(g, 2, 1, 140, 64, dtype=dtype).expand(-1, 3, -1, -1) for _ in range(2))
    m = (torch.rand(1, 140, generator=g, device="cuda") < 0.6).expand(2, -1)
    _check_all(q, k, v, do, 0.125, None, m)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("loss", ["sum", "mean over queries", "one head"])
def test_gradients_that_arrive_broadcast(dtype, loss):
    q, k, v, _ = (t.detach().clone().requires_grad_() for t in _inputs(dtype, 2, 4, 2, 20, 60))
    w = torch.randn(2, 4, 64, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(dtype)
    o = api.cross_attention(q, k, v)
    if loss == "sum":
        o.sum().backward()
        do = torch.ones_like(o)
    elif loss == "mean over queries":     # rows of dO with a stride of 0
        (o.sum(2) * w).sum().backward()
        do = w[:, :, None].expand_as(o)
    else:
        o[:, 1].sum().backward()
        do = torch.zeros_like(o)
        do[:, 1] = 1
    want = cross(q.detach(), k.detach(), v.detach(), 0.125, None, None, do, o.detach())
    for name, t in (("dQ", q), ("dK", k), ("dV", v)):
        check(name, t.grad, want[name])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(40, 2, 2, 150, 260), (6, 24, 2, 40, 700), (3, 12, 12, 1, 5000), (50, 12, 4, 6, 90), (2, 32, 2, 1, 300)],
                         ids=lambda s: "x".join(map(str, s)))
def test_more_units_than_the_gpu_holds(dtype, size):
    # several units a block, of both kinds in the backward, some without keys; rows of shared heads from 6 to 18
    q, k, v, do = _inputs(dtype, *size, seed=37)
    n, _ = _masks("len", size[0], size[4], seed=3)
    n[size[0] // 2] = 0
    _check_all(q, k, v, do, 0.125, n)


def test_gpu_refusals():
    q, k, v, do = _inputs(BF16, 2, 4, 2, 5, 9)
    with pytest.raises(ValueError, match="contiguous rows"):
        api.cross_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, 0.125)
    with pytest.raises(ValueError, match="kv_len"):
        api.cross_fwd(q, k, v, 0.125, kv_len=torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="kv_len"):
        api.cross_fwd(q, k, v, 0.125, kv_len=torch.ones(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="key_mask"):
        api.cross_fwd(q, k, v, 0.125, key_mask=torch.ones(2, 8, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError, match="key_mask"):
        api.cross_fwd(q, k, v, 0.125, key_mask=torch.ones(2, 9, device="cuda"))
    with pytest.raises(ValueError, match="dtype"):
        api.cross_fwd(q, k.float(), v, 0.125)
    with pytest.raises(api.FibattError, match="divide"):
        api.cross_fwd(q[:, :3], k, v, 0.125)
    with pytest.raises(api.FibattError, match=">= 1"):
        api.cross_fwd(q, k[:, :, :0], v[:, :, :0], 0.125)
    with pytest.raises(api.FibattError, match="overlap"):
        api.cross_fwd(q, k, v, 0.125, O=torch.empty(2, 1, 5, 64, dtype=BF16, device="cuda").expand(-1, 4, -1, -1))
    o, lse = api.cross_fwd(q, k, v, 0.125)
    with pytest.raises(api.FibattError, match="workspace"):
        api.cross_bwd(q, k, v, o, lse, do, 0.125, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_workspaces_and_streams_of_other_places_are_refused():
    q, k, v, do = _inputs(BF16, 2, 4, 2, 5, 9)
    o, lse = api.cross_fwd(q, k, v, 0.125)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        api.cross_bwd(q, k, v, o, lse, do, 0.125, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(TypeError, match="workspace"):
        api.cross_bwd(q, k, v, o, lse, do, 0.125, workspace=1 << 20)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        api.cross_bwd(q, k, v, o, lse, do, 0.125, workspace=torch.empty(1 << 20, 2, dtype=torch.uint8, device="cuda")[:, 0])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 6, 2, 50, 150), (1, 9, 3, 33, 300), (2, 10, 2, 1, 70)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("bad", [math.nan, 1e6])
def test_other_groups_queries_reach_no_gradient(dtype, size, bad):
    # a tile of query rows may end behind its group's last head
    q, k, v, do = _inputs(dtype, *size, layout="bhnd", seed=41)
    G = size[1] // size[2]
    want = _run(q, k, v, do, 0.125)
    q, do = q.clone(), do.clone()
    q[:, G:] = bad
    do[:, G:] = bad
    got = _run(q, k, v, do, 0.125)
    for name, n in (("O", G), ("LSE", G), ("dQ", G), ("dK", 1), ("dV", 1)):
        assert torch.equal(got[name][:, :n], want[name][:, :n]), name


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 40, 200])
def test_nan_in_attended_places_reaches_its_head(dtype, Nq):
    q, k, v, do = _inputs(dtype, 2, 4, 2, Nq, 150, layout="bhnd", seed=43)
    want = _run(q, k, v, do, 0.125)
    k[0, 0, 5, 3] = math.nan
    got = _run(q, k, v, do, 0.125)
    for name, n in (("O", 2), ("LSE", 2), ("dQ", 2), ("dK", 1), ("dV", 1)):
        assert bool(got[name][0, :n].isnan().all()), name
        assert torch.equal(got[name][0, n:], want[name][0, n:]) and torch.equal(got[name][1], want[name][1]), name


def test_gradients_of_gradients_are_refused():
    q, k, v, _ = (t.detach().clone().requires_grad_() for t in _inputs(F32, 1, 2, 2, 5, 9))
    dq, = torch.autograd.grad(api.cross_attention(q, k, v).square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dq.sum().backward()


@pytest.mark.parametrize("size", [(110, 6, 6, 20, 200), (60, 8, 8, 130, 300), (90, 6, 2, 50, 140)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("mask", ["none", "len", "both"])
def test_blocks_that_walk_over_their_units(size, mask):
    q, k, v, do = _inputs(BF16, *size, seed=47)
    n, m = _masks(mask, size[0], size[4], seed=5)
    if n is not None:
        n[size[0] // 3:size[0] // 2] = 0       # runs of units without keys
    _check_all(q, k, v, do, 0.125, n, m)


@pytest.mark.parametrize("Nk", [3, 4, 7, 16, 40, 128, 200])
@pytest.mark.parametrize("mask", ["none", "mask"])
def test_gradients_of_few_keys_have_two_roundings(Nk, mask):
    # dS and the result are each rounded once to 16 bits: at most 2^-8 of the value, uniform below
    # that, so 2^-8 / sqrt(3) in the mean square; two independent ones are sqrt(2) of it
    q, k, v, do = _inputs(BF16, 8, 4, 4, 60, Nk, layout="bhnd", seed=53)
    m = None
    if mask == "mask":
        m = torch.ones(8, Nk, dtype=torch.bool, device="cuda")
        m[:, ::3] = False
    got = _run(q, k, v, do, 0.125, None, m)
    want = cross(q, k, v, 0.125, None, m, do, got["O"])
    x, y, z, w = (t.double() for t in (q, k, v, do))
    s = 0.125 * x @ y.transpose(-1, -2)
    if m is not None:
        s = s.masked_fill(~m[:, None, None], -math.inf)
    p, dp = s.softmax(-1), w @ z.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    for name, exact in (("dQ", 0.125 * ds @ y), ("dK", 0.125 * ds.transpose(-1, -2) @ x)):
        check(name, got[name], want[name])
        err = float((got[name].double() - exact).norm() / exact.norm())
        assert err <= math.sqrt(2 / 3) * 2.0 ** -8, (name, err)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1, 30, 9000), (1, 2, 1, 9000, 20), (2, 6, 2, 40, 16385), (1, 4, 1, 2000, 300), (4, 4, 4, 100, 5000)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("mask", ["none", "len"])
def test_gradients_of_few_rows_on_many(dtype, size, mask):
    # one side's units walk over hundreds of tiles, the other's over one
    q, k, v, do = _inputs(dtype, *size, seed=59)
    n = None if mask == "none" else torch.full((size[0],), size[4] * 2 // 3, dtype=torch.int32, device="cuda")
    _check_all(q, k, v, do, 0.125, n)


@pytest.mark.parametrize("keys", [3, 4, 7, 8, 9, 64])
@pytest.mark.parametrize("Nk", [90, 128, 600, 1569])
@pytest.mark.parametrize("mask", ["none", "mask"])
def test_padding_does_not_cost_the_gradients_of_short_sequences_their_digits(keys, Nk, mask):
    # as above: two roundings of 2^-8 / sqrt(3), however long the tensors are
    q, k, v, do = _inputs(BF16, 8, 4, 2, 60, Nk, layout="bhnd", seed=53)
    n = torch.full((8,), keys, dtype=torch.int32, device="cuda")
    n[1::2] = Nk                    # next to sequences with all keys
    m, at = None, torch.arange(keys, device="cuda")
    if mask == "mask":
        m = torch.ones(8, Nk, dtype=torch.bool, device="cuda")
        m[:, 1::3] = False
        at = at[at % 3 != 1]
    got = _run(q, k, v, do, 0.125, n, m)
    want = cross(q, k, v, 0.125, n, m, do, got["O"])
    for name in got:
        check(name, got[name], want[name])
    x, y, z, w = (t[::2].double() for t in (q, k, v, do))
    y, z = (t[:, :, at].repeat_interleave(2, 1) for t in (y, z))
    p, dp = (0.125 * x @ y.transpose(-1, -2)).softmax(-1), w @ z.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dk = (0.125 * ds.transpose(-1, -2) @ x).view(4, 2, 2, len(at), 64).sum(2)
    for name, g, exact in (("dQ", got["dQ"][::2], 0.125 * ds @ y), ("dK", got["dK"][::2][:, :, at], dk)):
        err = float((g.double() - exact).norm() / exact.norm())
        assert err <= math.sqrt(2 / 3) * 2.0 ** -8, (name, err)


@pytest.mark.parametrize("size", [(40, 1, 1, 1, 70), (70, 1, 1, 3, 200), (9, 2, 1, 5, 1500), (3, 3, 3, 40, 3000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_sequences_of_few_and_of_many_keys_side_by_side(size):
    # sequences shorter than a block of the backward's first kernel, with none to all keys
    B, Nk = size[0], size[4]
    q, k, v, do = _inputs(BF16, *size, seed=61)
    g = torch.Generator(device="cuda").manual_seed(6)
    n = torch.randint(0, Nk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[::3] = torch.randint(0, 66, (len(n[::3]),), generator=g, device="cuda", dtype=torch.int32)
    share = torch.tensor([0.0, 0.01, 0.05, 0.5, 1.0], device="cuda")[torch.arange(B, device="cuda") % 5]
    m = torch.rand(B, Nk, generator=g, device="cuda") < share[:, None]
    for lens, mask in ((n, None), (None, m), (n, m)):
        _check_all(q, k, v, do, 0.125, lens, mask)
