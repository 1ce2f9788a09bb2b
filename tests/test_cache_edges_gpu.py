"""The paged 8-bit cache at the ends of its ranges: queries before the sequence, each in a call of its
own with the error word that it leaves; values up to the types' largest, which come back finite."""
import math

import pytest
import torch

from cache_ref import attend, decode, nearest
from test_cache_gpu import _cache, _error, _filled, _int32, _rand, _table
from window_ref import check, seen_of
from sparse_head_self_gb300 import api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


@TYPES
@pytest.mark.parametrize("start,count,word", [
    ((-25, 98), None, 16), ((-30, 98), None, 16), ((-2 ** 31, 98), None, 16), ((-1, 98), (1, 30), 16), ((98, 98), None, 0),
    ((-25, 98), (0, 30), 0), ((0, 98), None, 0), ((99, 98), None, 16), ((99, 98), (29, 30), 0), ((2 ** 31 - 1, 98), (0, 30), 0)], ids=str)
@pytest.mark.parametrize("Hq", [2, 1])
def test_queries_outside_the_table_are_reported(dtype, start, count, word, Hq):
    g = torch.Generator(device="cuda").manual_seed(12)
    cache, table, k, v = _filled(g, 2, 1, [128, 128], 2, dtype)
    q = _rand(g, 2, Hq, 30, 64, dtype=dtype)
    n = None if count is None else _int32(*count)
    o, lse = api.cache_fwd(q, cache, table, _int32(*start), 0.125, count=n)
    assert _error() == word
    seen = seen_of(2, 30, 128, None, 0, _int32(*start))
    if count is not None:
        seen = seen & (torch.arange(30, device="cuda") < n[:, None])[..., None]
    want = attend(q, k, v, 0.125, seen)
    check("O", o, want["O"])
    check("LSE", lse, want["LSE"])
    none = ~seen.any(2)
    assert bool((o.transpose(1, 2)[none] == 0).all()) and bool((lse.transpose(1, 2)[none] == -math.inf).all())


@TYPES
def test_the_largest_values_come_back_finite(dtype):
    # at the largest scale, 2^120, the largest value that 16 and 32 bits hold is the 240th multiple of it (an
    # infinity is the 448th, as at every scale)
    most = torch.finfo(dtype).max
    for top in (2.9e38, 448.0 * 2.0 ** 119, 3e38, 240.0 * 2.0 ** 120, 247.0 * 2.0 ** 120, 248.0 * 2.0 ** 120, 3.3e38, most):
        for odd in (0.0, math.inf, -math.inf, math.nan):
            x = torch.linspace(-1.0, 1.0, 40 * 64, dtype=torch.float64).view(1, 1, 40, 64) * top
            K = x.clamp(-most, most).to(dtype).clamp(-most, most).cuda()
            K[0, 0, 1, 2] = odd
            V = (-K).flip(2).contiguous()
            cache, table = _cache(1, 1, junk=False), _table(1, 1, 1)
            api.cache_store(cache, table, K, V)
            for kind, src in enumerate((K, V)):
                src = src[0, 0].double().cpu()
                size = float(src[src.isfinite()].abs().max())
                scale = 2.0 ** 119 if size <= 448.0 * 2.0 ** 119 else 2.0 ** 120
                assert float(cache.scales[0, 0, kind]) == scale, (top, odd)
                want = decode(nearest(src / scale))
                if scale == 2.0 ** 120:
                    want = torch.where(src.isfinite(), want.clamp(-240.0, 240.0), want)
                for dt in (F32, BF16):
                    got = api.cache_load(cache, table, 40, dtype=dt)[kind][0, 0].double().cpu()
                    assert torch.equal(got.isnan(), src.isnan()) and bool(got[src.isfinite()].isfinite().all()), (top, odd)
                    clear = lambda t: t.float().nan_to_num(-7.0, math.inf, -math.inf)  # noqa: E731
                    assert torch.equal(clear(got), clear(want * scale)), (top, odd)


def test_a_pages_older_tokens_at_the_largest_scale():
    K = torch.full((1, 1, 2, 64), 448.0 * 2.0 ** 119, device="cuda")
    K[0, 0, 1] = torch.finfo(F32).max
    cache, table = _cache(1, 1, junk=False), _table(1, 1, 1)
    for i in range(2):
        api.cache_store(cache, table, K[:, :, i:i + 1], K[:, :, i:i + 1], _int32(i))
    for t in api.cache_load(cache, table, 2, dtype=F32):
        assert t[0, 0].tolist() == [[224.0 * 2.0 ** 120] * 64, [240.0 * 2.0 ** 120] * 64]
