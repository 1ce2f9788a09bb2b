"""The library's auxiliary tools on the attention over a window and the 8-bit
cache: the bounds-checked build on a selection of their tests, in a child process
(the binding loads one library per process), and the per-kernel timing print."""
import os
import re
import subprocess
import sys

import pytest
import torch

from test_cross_gpu import _inputs
from sparse_head_self_gb300 import api

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checks_build_runs_the_window_and_the_cache_clean():
    env = dict(os.environ, FIBATT_CHECKS="1")
    env.pop("FIBATT_PROFILE", None)
    sel = ("values_and_gradients or units or other_groups or rows_are_written or starts_outside or long_walk "
           "or few_keys or chunk_by_chunk or attention or prefix or do_not_have")
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_window_gpu.py", "tests/test_window_front_gpu.py",
                        "tests/test_cache_gpu.py", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider", "-k", sel], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=1800)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert "libfibatt checks" not in r.stderr, tail
    assert re.search(r"\d+ passed", r.stdout), tail


def test_profile_prints_each_kernel(capfd, monkeypatch):
    q, k, v, do = _inputs(torch.bfloat16, 1, 4, 2, 300, 300)
    cache, table = api.Cache.new(5, 2), torch.arange(5, dtype=torch.int32, device="cuda")[None]
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("FIBATT_PROFILE", "1")
    capfd.readouterr()
    o, lse = api.window_fwd(q, k, v, 0.125, 100)
    api.window_bwd(q, k, v, o, lse, do, 0.125, 100)
    api.cache_store(cache, table, k, v)
    api.cache_load(cache, table, 300)
    api.cache_fwd(q[:, :, :2], cache, table, start, 0.125)
    torch.cuda.synchronize()
    err = capfd.readouterr().err
    for call, kernel in (("fibatt_window_fwd", "cross_fwd_mma_kernel"), ("fibatt_window_bwd", "window_parts_kernel"),
                         ("fibatt_window_bwd", "cross_bwd_mma_kernel"), ("fibatt_cache_store", "cache_store_kernel"),
                         ("fibatt_cache_load", "cache_load_kernel"), ("fibatt_cache_fwd", "cache_fwd_kernel")):
        assert re.search(rf"libfibatt profile: {call} .*{kernel}", err), (call, kernel, err)
