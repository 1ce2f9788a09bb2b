"""A query that attends keys and brings a NaN or an infinity, its own or its gradient's: the
gradients of the keys that it attends have it, those of keys that nobody attends are
zeros all the same, next to it in a tile or not; other queries, heads and sequences have nothing of it."""
import math

import pytest
import torch

from test_cross_gpu import _inputs
from test_cross_gpu import _run as _run_cross
from test_window_gpu import _run, _seen
from sparse_head_self_gb300 import api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def _ids(s):
    return "x".join(map(str, s))


def _int32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@TYPES
@pytest.mark.parametrize("size,band,length", [
    ((3, 4, 2, 300, 300), (40, 3), 100),        # the sinks' tile ends with keys that nobody attends
    ((1, 8, 2, 1000, 1000), (128, 4), 100), ((1, 8, 2, 1000, 1000), (128, 4), 950), ((2, 4, 2, 1500, 1500), (64, 130), 200),
    ((3, 4, 2, 300, 300), (130, 0), 170), ((3, 4, 2, 300, 300), (None, 0), 290), ((2, 2, 2, 70, 300), (None, 0), 200),
    ((2, 4, 1, 5, 300), (40, 3), 100), ((40, 2, 2, 150, 260), (150, 4), 90), ((1, 2, 1, 40, 2000), (None, 0), 1900),
    ((1, 2, 1, 40, 2000), (500, 4), 100), ((8, 4, 4, 60, 60), (3, 0), 37), ((8, 4, 2, 60, 60), (8, 1), 9)], ids=str)
@pytest.mark.parametrize("where,bad", [("dO", math.nan), ("dO", math.inf), ("Q", math.nan)])
def test_window(dtype, size, band, length, where, bad):
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(dtype, *size, layout="bhnd", seed=71)
    n = torch.full((B,), Nk, dtype=torch.int32, device="cuda")
    n[0] = length
    how = {"window": band[0], "sinks": band[1], "kv_len": n}
    if Nq < Nk:
        how["q_start"] = n - Nq
    j = Nq - 1 if Nq < Nk else length - 1       # the sequence's last query
    seen = _seen(q, k, how)[0]
    clean = _run(q, k, v, do, 0.125, **how)
    if where == "Q":
        q = q.clone()
        q[0, 0, j, 5] = bad
    else:
        do = do.clone()
        do[0, 0, j, 5] = bad
    got = _run(q, k, v, do, 0.125, **how)
    dead = ~seen.any(0)
    assert bool(dead.any()) and bool(seen[j].any())
    for name in ("dK", "dV"):
        assert bool((got[name][0, :, dead] == 0).all()), name
        assert torch.equal(got[name][0, 1:], clean[name][0, 1:]) and torch.equal(got[name][1:], clean[name][1:]), name
        near = torch.nn.functional.max_pool1d(seen[j].float()[None], 511, 1, 255)[0] > 0
        assert torch.equal(got[name][0, 0, ~near], clean[name][0, 0, ~near]), name
    assert not bool(got["dV"][0, 0, seen[j]][:, 5].isfinite().any())
    for name in ("O", "LSE", "dQ"):
        if name != "dQ" and where != "Q":
            assert torch.equal(got[name], clean[name]), name
            continue
        assert not bool(got[name][0, 0, j].isfinite().all()), name
        got[name][0, 0, j] = clean[name][0, 0, j]
        assert torch.equal(got[name], clean[name]), name


@TYPES
@pytest.mark.parametrize("size", [(2, 4, 2, 70, 300), (2, 4, 2, 1, 300), (2, 4, 1, 5, 40), (1, 2, 1, 40, 2000), (40, 2, 2, 130, 300)],
                         ids=_ids)
@pytest.mark.parametrize("masked", [False, True], ids=["len", "mask"])
@pytest.mark.parametrize("where,bad", [("dO", math.nan), ("dO", math.inf), ("Q", math.nan)])
def test_cross(dtype, size, masked, where, bad):
    B, Hq, Hkv, Nq, Nk = size
    q, k, v, do = _inputs(dtype, *size, layout="bhnd", seed=73)
    n = torch.full((B,), Nk - Nk // 5, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    m = torch.rand(B, Nk, device="cuda", generator=g) < 0.7 if masked else None
    keep = torch.arange(Nk, device="cuda") < n[0]
    if masked:
        keep = keep & m[0]
    clean = _run_cross(q, k, v, do, 0.125, n, m)
    (q if where == "Q" else do)[0, 0, Nq // 2, 5] = bad
    got = _run_cross(q, k, v, do, 0.125, n, m)
    for name in ("dK", "dV"):
        assert bool((got[name][0, :, ~keep] == 0).all()), name
        assert torch.equal(got[name][0, 1:], clean[name][0, 1:]) and torch.equal(got[name][1:], clean[name][1:]), name
    assert not bool(got["dV"][0, 0, keep][:, 5].isfinite().any())
    got["dQ"][0, 0, Nq // 2] = clean["dQ"][0, 0, Nq // 2]
    assert torch.equal(got["dQ"], clean["dQ"])


def test_autograd_of_a_padded_batch_with_a_nan_loss():
    # the padding's gradients, which a packed projection sums with the others', stay zeros
    q, k, v, _ = (t.detach().clone().requires_grad_() for t in _inputs(BF16, 2, 8, 2, 600, 600))
    n = _int32(90, 600)
    o = api.window_attention(q, k, v, window=50, sinks=4, kv_len=n)
    (o[0, :, 89] * math.nan).sum().backward()
    assert bool((k.grad[0, :, 90:] == 0).all()) and bool((v.grad[0, :, 90:] == 0).all())
    assert bool(v.grad[0, :, 45:90].isnan().all())
