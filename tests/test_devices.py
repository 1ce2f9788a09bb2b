"""What the library keeps about a device is kept for each device: the cache on
the CPU, and calls that want clusters of 16 on a second GPU where there is one."""
import os
import subprocess

import pytest
import torch

from sparse_head_self_gb300.build import CSRC

PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
#include <initializer_list>
int main() {
    fibatt::PerDevice known;
    int asked[80] = {}, wrong = 0;
    const auto answer = [&](int dev) { return known.get(dev, [&] { ++asked[dev + 1]; return 100 + dev; }); };
    for (int turn = 0; turn < 3; ++turn)
        for (int dev : {0, 1, 7, 63, 64, 70, -1}) wrong += answer(dev) != 100 + dev;
    // each device is asked itself, once; those that are not kept, each time
    for (int dev : {0, 1, 7, 63}) wrong += asked[dev + 1] != 1;
    for (int dev : {64, 70, -1}) wrong += asked[dev + 1] != 3;
    printf("%d\n", wrong);
    return wrong != 0;
}
"""


def test_answers_are_kept_for_each_device(tmp_path):
    src, exe = tmp_path / "per_device.cpp", tmp_path / "per_device"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "0\n"


def test_every_request_for_large_clusters_is_behind_that_cache():
    # the permission for more than eight CTAs belongs to the current device: it is set in one place,
    # and what calls that place goes through PerDevice
    text = {f: open(os.path.join(CSRC, f)).read() for f in sorted(os.listdir(CSRC))}
    assert [f for f, t in text.items() if "NonPortableClusterSizeAllowed" in t] == ["cross.h"]
    for f, t in text.items():
        if f != "cross.h" and "clusters_held<" in t.replace("held_clusters<", ""):
            assert "static PerDevice" in t, f


@pytest.mark.gpu
@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one GPU")
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_few_heads_on_many_keys_on_two_devices(dtype):
    from sparse_head_self_gb300 import api
    got = []
    for index in (0, 1):
        g = torch.Generator().manual_seed(0)
        q, k, v, do = (torch.randn(1, 1, n, 64, generator=g).to(dtype).to(f"cuda:{index}") for n in (100, 16385, 16385, 100))
        o, lse = api.cross_fwd(q, k, v, 0.125)
        got.append([t.cpu() for t in (o, lse, *api.cross_bwd(q, k, v, o, lse, do, 0.125))])
    for a, b in zip(*got):
        assert torch.equal(a, b)
