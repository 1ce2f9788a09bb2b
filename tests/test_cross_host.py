"""Host-side tests of the query/key norm and the cross attention (no GPU
needed): every refusal of the two C calls and of their Python entry points,
each before anything is launched, and the rotary angle helpers."""
import math

import pytest
import torch

from sparse_head_self_gb300 import _native, api
from sparse_head_self_gb300.build import build_all

INVALID, UNSUPPORTED, CUDA = 1, 2, 3
P = 1 << 20   # a pointer that is never followed: every call below fails its checks first


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_all()
    yield


def _heads(ptr=P, b=64 * 9 * 2, h=64 * 9, n=64):
    return _native.HEADS.pack(ptr or 0, b, h, n)


def _cross_desc(**kw):
    d = {**dict(B=2, Hq=4, Hkv=2, Nq=9, Nk=9, D=64, dtype=1, scale=0.125, kv_len=0, key_mask=0, key_mask_stride_b=0), **kw}
    return _native.CROSS.pack(*d.values())


def _cross(bwd=False, q=None, k=None, v=None, o=None, lse=P, do=None, dq=None, dk=None, dv=None, ws=P, ws_bytes=1 << 20,
           **kw):
    L = _native.lib()
    d = _cross_desc(**kw)
    r = [x or _heads() for x in (q, k, v, o)]
    if not bwd:
        return L.fibatt_cross_fwd(d, *r, lse, None)
    g = [x or _heads() for x in (do, dq, dk, dv)]
    return L.fibatt_cross_bwd(d, *r, lse, *g, ws, ws_bytes, None)


@pytest.fixture
def _no_launch(monkeypatch):
    """A call that passes its checks stops at the injected launch failure."""
    monkeypatch.setenv("FIBATT_FAULT", "launch")


@pytest.mark.parametrize("bwd", [False, True])
def test_cross_refusals(bwd, _no_launch):
    def st(**kw):
        return _cross(bwd, **kw)

    assert st() == CUDA   # nothing wrong with the arguments: it would have launched
    for n in ("B", "Hq", "Hkv", "Nq", "Nk"):
        assert st(**{n: 0}) == INVALID, n
        assert st(**{n: -3}) == INVALID, n
    assert st(Hkv=3) == INVALID and "divide" in _native.lib().fibatt_last_error().decode()
    assert st(D=128) == UNSUPPORTED
    assert st(dtype=5) == UNSUPPORTED
    for s in (math.inf, math.nan):
        assert st(scale=s) == INVALID
    for s in (0.0, -0.5):
        assert st(scale=s) == CUDA
    assert st(kv_len=P + 2) == INVALID
    assert st(key_mask=P, key_mask_stride_b=-1) == INVALID
    assert st(key_mask=P + 1, key_mask_stride_b=9) == CUDA
    for name in ("q", "k", "v", "o"):
        assert st(**{name: _heads(ptr=None)}) == INVALID
        assert st(**{name: _heads(ptr=P + 8)}) == INVALID
        assert st(**{name: _heads(n=68)}) == INVALID      # 136 bytes between the rows
        assert st(**{name: _heads(h=-64)}) == INVALID
        assert st(**{name: _heads(n=0)}) == INVALID       # no broadcast rows
        assert st(**{name: _heads(b=1 << 39)}) == INVALID
    for name in ("q", "k", "v"):
        assert st(**{name: _heads(b=0)}) == CUDA          # broadcast inputs are read
        assert st(**{name: _heads(h=0)}) == CUDA
    for name in ("dq", "dk", "dv") if bwd else ("o",):
        for s in ("b", "h", "n"):
            assert st(**{name: _heads(**{s: 0})}) == INVALID, (name, s)
        assert st(**{name: _heads(n=32)}) == INVALID
    assert st(lse=None) == INVALID
    assert st(lse=P + 2) == INVALID
    assert st(B=1 << 20, Nq=1 << 18) == INVALID           # 2^34 blocks
    if bwd:
        assert st(ws=None) == INVALID
        need = _native.lib().fibatt_cross_bwd_workspace_bytes(_cross_desc())
        assert st(ws_bytes=need - 1) == INVALID and st(ws_bytes=need) == CUDA
        assert st(do=_heads(ptr=P + 4)) == INVALID


def test_cross_workspace_size():
    L = _native.lib()
    assert L.fibatt_cross_bwd_workspace_bytes(_cross_desc()) >= 2 * 4 * 9 * 8
    assert L.fibatt_cross_bwd_workspace_bytes(_cross_desc(B=0)) == 0
    assert L.fibatt_cross_bwd_workspace_bytes(None) == 0


def _norm(bwd=False, x=P, sb=9 * 8 * 64, sn=8 * 64, q=P, k=P, v=P, dx=P, dsb=9 * 8 * 64, dsn=8 * 64, ws=P, ws_bytes=1 << 20,
          dw=P, **kw):
    L = _native.lib()
    d = {**dict(B=2, N=9, Hq=4, Hk=2, Hv=2, D=64, dtype=1, q_weight=P, k_weight=P, eps=1e-6, rot_dims=64, interleaved=0,
                cos=P, sin=P, table_len=9, positions=0, positions_stride_b=0), **kw}
    d = _native.QK_NORM.pack(*(0 if f is None else f for f in d.values()))
    if not bwd:
        return L.fibatt_qk_norm_fwd(d, x, sb, sn, q, k, v, None)
    return L.fibatt_qk_norm_bwd(d, x, sb, sn, q, k, v, dx, dsb, dsn, dw, dw, ws, ws_bytes, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_qk_norm_refusals(bwd, _no_launch):
    def st(**kw):
        return _norm(bwd, **kw)

    assert st() == CUDA
    for kw in (dict(B=0), dict(N=0), dict(Hq=-1), dict(Hq=0, Hk=0, Hv=0), dict(eps=-1e-6), dict(eps=math.nan),
               dict(eps=math.inf), dict(rot_dims=8), dict(rot_dims=80), dict(rot_dims=-16), dict(cos=None),
               dict(sin=None), dict(cos=P + 4), dict(table_len=8), dict(table_len=0, positions=P),
               dict(positions=P + 2), dict(positions=P, positions_stride_b=-1), dict(q_weight=P + 2),
               dict(x=None), dict(x=P + 8), dict(sn=8 * 64 + 4), dict(sb=-64), dict(q=None), dict(k=None), dict(v=None),
               dict(q=P + 8), dict(B=1 << 16, N=1 << 15, positions=P)):
        assert st(**kw) == INVALID, kw
    assert st(D=32) == UNSUPPORTED
    assert st(dtype=9) == UNSUPPORTED
    # what a call does not use may be missing
    assert st(q_weight=None, k_weight=None) == CUDA
    assert st(rot_dims=0, cos=None, sin=None, table_len=0) == CUDA
    assert st(Hq=0, q=None) == CUDA
    assert st(positions=P, table_len=1) == CUDA
    assert st(eps=0.0) == CUDA
    if bwd:
        for kw in (dict(dx=None), dict(dx=P + 8), dict(dsn=8 * 64 - 8), dict(dsb=0), dict(ws=None), dict(ws=P + 8),
                   dict(ws_bytes=1024), dict(dw=P + 2)):
            assert st(**kw) == INVALID, kw
        assert st(dw=None) == CUDA


def test_injected_argument_fault(monkeypatch):
    monkeypatch.setenv("FIBATT_FAULT", "arg")
    for st in (_cross(), _cross(True), _norm(), _norm(True)):
        assert st == INVALID
        assert "injected" in _native.lib().fibatt_last_error().decode()


def test_python_entry_points_reject_what_they_cannot_take():
    q, x = torch.zeros(1, 2, 3, 64), torch.zeros(1, 3, 6 * 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.cross_fwd(q, q, q, 0.125)
    with pytest.raises(ValueError, match="CUDA"):
        api.qk_norm_fwd(x, (2, 2, 2))
    with pytest.raises(ValueError, match="B, H, N, D"):
        api.cross_fwd(q[0], q, q, 0.125)
    with pytest.raises(ValueError, match="dtype"):
        api.cross_fwd(q.half(), q.half(), q.half(), 0.125)
    with pytest.raises(ValueError, match="dtype"):
        api.qk_norm_fwd(x.double(), (2, 2, 2))
    with pytest.raises(ValueError, match="B, N"):
        api.qk_norm_fwd(x[0], (2, 2, 2))


def test_packed_structures_are_as_c_lays_them_out(tmp_path):
    # sizes and field offsets of the header's structures against the packed formats'
    import os
    import subprocess

    fields = {
        "fibatt_heads": (_native.HEADS, ["ptr", "stride_b", "stride_h", "stride_n"]),
        "fibatt_cross": (_native.CROSS, ["B", "Hq", "Hkv", "Nq", "Nk", "D", "dtype", "scale", "kv_len", "key_mask",
                                         "key_mask_stride_b"]),
        "fibatt_qk_norm": (_native.QK_NORM, ["B", "N", "Hq", "Hk", "Hv", "D", "dtype", "q_weight", "k_weight", "eps",
                                             "rot_dims", "interleaved", "cos", "sin", "table_len", "positions",
                                             "positions_stride_b"]),
    }
    lines = []
    for name, (_, names) in fields.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f in names]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdint.h>\n#include <stdio.h>\n#include "fibatt.h"\n'
                   "int main(void) { " + " ".join(lines) + " return 0; }\n")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["gcc", "-I", os.path.dirname(_native.HEADER), "-I", cuda, "-o", str(tmp_path / "layout"), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()]
    for name, (fmt, names) in fields.items():
        size, offsets, got = got[0], got[1:1 + len(names)], got[1 + len(names):]
        assert fmt.size == size, name
        for i in range(len(names)):
            # a value in field i alone: its first byte stands at the field's offset
            blob = fmt.pack(*(1.0 if names[k] in ("scale", "eps") and k == i else int(k == i) for k in range(len(names))))
            at = next(p for p, x in enumerate(blob) if x)
            want = offsets[i] + (2 if names[i] in ("scale", "eps") else 0)      # 1.0f is 00 00 80 3f
            assert at == want, (name, names[i])


def test_rotary_angles():
    a = api.rotary_angles(7, 32, 10000.0)
    assert a.shape == (7, 16) and a.dtype == torch.float64
    for p in (0, 3, 6):
        for i in (0, 5, 15):
            assert a[p, i].item() == pytest.approx(p * 10000.0 ** (-2 * i / 32), rel=1e-12)
    b = api.rotary_angles_2d(3, 5, 64, 100.0)
    assert b.shape == (15, 32)
    for r in range(3):
        for c in range(5):
            for i in range(16):
                f = 100.0 ** (-2 * i / 32)
                assert b[r * 5 + c, i].item() == pytest.approx(r * f, rel=1e-12)
                assert b[r * 5 + c, 16 + i].item() == pytest.approx(c * f, rel=1e-12)
    cos, sin = api.rotary_tables(a)
    assert cos.dtype == torch.float32 and torch.equal(cos, a.cos().float()) and torch.equal(sin, a.sin().float())
    with pytest.raises(ValueError, match="pairs"):
        api.rotary_tables(torch.zeros(4, 5))
