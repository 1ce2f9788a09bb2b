"""Host-side tests of the attention over a window (no GPU needed): every refusal of
the two C calls and of their Python entry points, each before anything is launched."""
import math
import os
import subprocess

import pytest
import torch

from sparse_head_self_gb300 import _native, api
from test_cross_host import CUDA, INVALID, P, UNSUPPORTED, _built, _heads, _no_launch  # noqa: F401


def _desc(**kw):
    d = {**dict(B=2, Hq=4, Hkv=2, Nq=9, Nk=9, D=64, dtype=1, scale=0.125, window=5, sinks=2, q_start=0, kv_len=0), **kw}
    return _native.WINDOW.pack(*d.values())


def _window(bwd=False, q=None, k=None, v=None, o=None, lse=P, do=None, dq=None, dk=None, dv=None, ws=P, ws_bytes=1 << 20,
            **kw):
    L = _native.lib()
    d = _desc(**kw)
    r = [x or _heads() for x in (q, k, v, o)]
    if not bwd:
        return L.fibatt_window_fwd(d, *r, lse, None)
    g = [x or _heads() for x in (do, dq, dk, dv)]
    return L.fibatt_window_bwd(d, *r, lse, *g, ws, ws_bytes, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_window_refusals(bwd, _no_launch):  # noqa: F811
    def st(**kw):
        return _window(bwd, **kw)

    assert st() == CUDA   # nothing wrong with the arguments: it would have launched
    for n in ("B", "Hq", "Hkv", "Nq", "Nk"):
        assert st(**{n: 0}) == INVALID, n
        assert st(**{n: -3}) == INVALID, n
    assert st(Hkv=3) == INVALID and "divide" in _native.lib().fibatt_last_error().decode()
    assert st(D=128) == UNSUPPORTED
    assert st(dtype=5) == UNSUPPORTED
    for s in (math.inf, math.nan):
        assert st(scale=s) == INVALID
    for w in (0, -1):
        assert st(window=w) == INVALID and "window" in _native.lib().fibatt_last_error().decode()
    assert st(window=1) == CUDA and st(window=2 ** 31 - 1, sinks=2 ** 31 - 1) == CUDA
    assert st(sinks=-1) == INVALID and "sinks" in _native.lib().fibatt_last_error().decode()
    assert st(kv_len=P + 2) == INVALID and st(q_start=P + 2) == INVALID
    assert st(Nq=10) == INVALID and "q_start" in _native.lib().fibatt_last_error().decode()
    assert st(Nq=10, q_start=P) == CUDA
    assert st(Nk=1 << 30, B=1) == INVALID and st(Nq=1 << 30, B=1, q_start=P) == INVALID
    for name in ("q", "k", "v", "o"):
        assert st(**{name: _heads(ptr=None)}) == INVALID
        assert st(**{name: _heads(ptr=P + 8)}) == INVALID
        assert st(**{name: _heads(n=68)}) == INVALID
    for name in ("q", "k", "v"):
        assert st(**{name: _heads(b=0)}) == CUDA          # broadcast inputs are read
    for name in ("dq", "dk", "dv") if bwd else ("o",):
        assert st(**{name: _heads(h=0)}) == INVALID, name
    assert st(lse=None) == INVALID and st(lse=P + 2) == INVALID
    assert st(B=1 << 20, Nq=1 << 18, Nk=1 << 18) == INVALID           # 2^34 blocks
    if bwd:
        assert st(ws=None) == INVALID
        need = _native.lib().fibatt_window_bwd_workspace_bytes(_desc())
        assert st(ws_bytes=need - 1) == INVALID and st(ws_bytes=need) == CUDA
        assert st(do=_heads(ptr=P + 4)) == INVALID


def test_window_workspace_size():
    L = _native.lib()
    assert L.fibatt_window_bwd_workspace_bytes(_desc()) >= 2 * 4 * 9 * 8
    assert L.fibatt_window_bwd_workspace_bytes(_desc(B=0)) == 0
    assert L.fibatt_window_bwd_workspace_bytes(None) == 0


def test_injected_argument_fault(monkeypatch):
    monkeypatch.setenv("FIBATT_FAULT", "arg")
    for st in (_window(), _window(True)):
        assert st == INVALID and "injected" in _native.lib().fibatt_last_error().decode()


def test_python_entry_points_reject_what_they_cannot_take():
    q = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.window_fwd(q, q, q, 0.125, 2)
    with pytest.raises(ValueError, match="B, H, N, D"):
        api.window_fwd(q[0], q, q, 0.125, 2)
    with pytest.raises(ValueError, match="dtype"):
        api.window_fwd(q.half(), q.half(), q.half(), 0.125, 2)


def layouts_agree(tmp_path, structs):
    """Sizes and offsets of the header's structures against the packed formats'; structs:
    {name: (format, [fields])}."""
    lines = []
    for name, (_, names) in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f in names]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdint.h>\n#include <stdio.h>\n#include "fibatt.h"\n'
                   "int main(void) { " + " ".join(lines) + " return 0; }\n")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["gcc", "-I", os.path.dirname(_native.HEADER), "-I", cuda, "-o", str(tmp_path / "layout"), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()]
    for name, (fmt, names) in structs.items():
        size, offsets, got = got[0], got[1:1 + len(names)], got[1 + len(names):]
        assert fmt.size == size, name
        for i, field in enumerate(names):
            # a value in field i alone: its first byte stands at the field's offset (1.0f is 00 00 80 3f)
            blob = fmt.pack(*(1.0 if f == "scale" and f == field else int(f == field) for f in names))
            assert next(p for p, x in enumerate(blob) if x) == offsets[i] + (2 if field == "scale" else 0), (name, field)


def test_the_packed_structure_is_as_c_lays_it_out(tmp_path):
    layouts_agree(tmp_path, {"fibatt_window": (_native.WINDOW, ["B", "Hq", "Hkv", "Nq", "Nk", "D", "dtype", "scale", "window",
                                                                "sinks", "q_start", "kv_len"])})
