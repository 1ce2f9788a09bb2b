"""The paged 8-bit cache at the ends of its ranges: queries before the sequence, each in a call of its
own with the error word that it leaves."""
import math

import pytest
import torch

from cache_ref import attend
from test_cache_gpu import _error, _filled, _int32, _rand
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
