"""Host-side tests of the paged 8-bit cache (no GPU needed): every refusal of its C
calls and of their Python entry points; where the kernels' blocks read and write,
computed by the same functions on the CPU; the reference's own 8-bit values."""
import math
import subprocess

import pytest
import torch

import cache_ref
from sparse_head_self_gb300 import _native, api
from sparse_head_self_gb300.build import CSRC
from test_cross_host import CUDA, INVALID, P, UNSUPPORTED, _built, _heads, _no_launch  # noqa: F401
from test_window_host import layouts_agree


def _desc(**kw):
    d = {**dict(B=2, Hkv=2, N=9, D=64, dtype=1, pages=7, table_len=3, data=P, scales=P, table=P, table_stride_b=3, start=0,
                count=0), **kw}
    return _native.CACHE.pack(*(0 if x is None else x for x in d.values()))


def _call(kind, k=None, v=None, q=None, o=None, lse=P, Hq=4, scale=0.125, window=5, sinks=2, **kw):
    L = _native.lib()
    d = _desc(**kw)
    if kind == "fwd":
        return L.fibatt_cache_fwd(d, Hq, scale, window, sinks, q or _heads(), o or _heads(), lse, None)
    return getattr(L, "fibatt_cache_" + kind)(d, k or _heads(), v or _heads(), None)


@pytest.mark.parametrize("kind", ["store", "load", "fwd"])
def test_cache_refusals(kind, _no_launch):  # noqa: F811
    def st(**kw):
        return _call(kind, **kw)

    assert st() == CUDA
    for n in ("B", "Hkv", "N", "pages", "table_len"):
        assert st(**{n: 0}) == INVALID, n
        assert st(**{n: -3}) == INVALID, n
    assert st(D=128) == UNSUPPORTED and st(dtype=5) == UNSUPPORTED
    for name, off in (("data", 8), ("scales", 4), ("table", 2)):
        assert st(**{name: None}) == INVALID, name
        assert st(**{name: P + off}) == INVALID, name
    assert st(start=P + 2) == INVALID and st(count=P + 2) == INVALID and st(start=P, count=P) == CUDA
    assert st(table_stride_b=-1) == INVALID and st(table_stride_b=0) == CUDA
    assert st(N=1 << 30) == INVALID and st(table_len=1 << 24) == INVALID
    assert st(B=1 << 20, Hkv=1 << 6, N=1 << 12) == INVALID
    for name in ("q", "o") if kind == "fwd" else ("k", "v"):
        assert st(**{name: _heads(ptr=None)}) == INVALID and st(**{name: _heads(ptr=P + 8)}) == INVALID
        assert st(**{name: _heads(n=68)}) == INVALID and st(**{name: _heads(n=0)}) == INVALID
        written = name == "o" or kind == "load"
        assert st(**{name: _heads(h=0)}) == (INVALID if written else CUDA), name
    if kind == "fwd":
        assert st(Hq=3) == INVALID and "divide" in _native.lib().fibatt_last_error().decode()
        assert st(Hq=0) == INVALID
        for s in (math.inf, math.nan):
            assert st(scale=s) == INVALID
        assert st(window=0) == INVALID and st(sinks=-1) == INVALID
        assert st(window=2 ** 31 - 1, sinks=2 ** 31 - 1) == CUDA
        assert st(lse=None) == INVALID and st(lse=P + 2) == INVALID


def test_injected_argument_fault(monkeypatch):
    monkeypatch.setenv("FIBATT_FAULT", "arg")
    for kind in ("store", "load", "fwd"):
        assert _call(kind) == INVALID and "injected" in _native.lib().fibatt_last_error().decode()


def test_python_entry_points_reject_what_they_cannot_take():
    q = torch.zeros(1, 2, 3, 64)
    cache, table = api.Cache.new(4, 2, "cpu"), torch.zeros(1, 2, dtype=torch.int32)
    assert cache.data.shape == (4, 2, 2, 4096) and cache.scales.shape == (4, 2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        api.cache_store(cache, table, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        api.cache_load(cache, table, 3)
    with pytest.raises(ValueError, match="CUDA"):
        api.cache_fwd(q, cache, table, None, 0.125)
    with pytest.raises(ValueError, match="B, H, N, D"):
        api.cache_store(cache, table, q[0], q[0])
    with pytest.raises(ValueError, match="B, H, N, D"):
        api.cache_fwd(q[0], cache, table, None, 0.125)


def test_the_packed_structure_is_as_c_lays_it_out(tmp_path):
    layouts_agree(tmp_path, {"fibatt_cache": (_native.CACHE, ["B", "Hkv", "N", "D", "dtype", "pages", "table_len", "data", "scales",
                                                              "table", "table_stride_b", "start", "count"])})


# The kernels' own index functions on the CPU: every table entry, page and row that a block touches is
# in its buffer, every token is some block's, and the walks meet just the tiles with keys that are seen.
PROGRAM = r"""
#include "cross_cache.h"
#include <cstdio>
#include <random>
#include <set>
#include <vector>
using namespace fibatt;
template <int T> int walks(const Band &w, int lo, int hi, int end) {
    const BandWalk<T> walk(w, lo, hi);
    std::set<int> want, got;
    for (int k = 0; k < end; ++k)
        for (int p = lo; p <= hi; ++p)
            if (w.sees(p, k)) want.insert(k / T);
    int wrong = 0;
    for (int i = 0; i < walk.n; ++i) wrong += !got.insert(walk.tile(i)).second;
    for (int t : want) wrong += !got.count(t);
    for (int t : got) wrong += t < 0 || t * T > hi;
    wrong += got.size() > want.size() + 1;      // (a tile may hold the window's start only in part)
    return wrong;
}
// From the oldest key on: every pair once, in a tile that is met once.
template <int T> int pairs(const Band &w, int lo, int hi, int end) {
    const KeyWalk<T> walk(w, lo, hi);
    std::set<std::pair<int, int>> got;
    int wrong = 0;
    for (int i = 0; i < walk.n; ++i) {
        const Band x = walk.band(w, i);
        const int k0 = walk.key(i);
        wrong += k0 < 0 || k0 > hi;
        for (int p = lo; p <= hi; ++p)
            for (int k = 0; k < T; k += 32)
                for (uint32_t m = keys_of(x, p, k0 + k); m; m &= m - 1) {
                    const int key = k0 + k + __builtin_ctz(m);
                    wrong += !got.insert({p, key}).second || !(keys_between(x, lo, hi, k0 + k) >> __builtin_ctz(m) & 1);
                }
        wrong += keys_of(x, -1, k0) != 0;
    }
    for (int p = lo; p <= hi; ++p)
        for (int k = 0; k < end; ++k) wrong += w.sees(p, k) != (bool)got.count({p, k});
    if (lo <= hi) wrong += walk.n > (w.sinks + T - 1) / T + (w.window + hi - lo) / T + 1;
    return wrong;
}
int main() {
    std::mt19937 r(1);
    const auto in = [&](int a, int b) { return a + (int)(r() % (unsigned)(b - a + 1)); };
    const int far[] = {-2147483647 - 1, -1000000, -64, -1, 0, 63, 64, 1000000, 2147483647};
    int wrong = 0;
    for (int turn = 0; turn < 20000; ++turn) {
        CacheArgs a = {};
        a.B = in(1, 4), a.Hkv = in(1, 3), a.N = in(1, 200), a.pages = in(1, 20), a.table_len = in(1, 6), a.table_sb = in(0, 1) * a.table_len;
        std::vector<int32_t> table(a.B * a.table_len), start(a.B), count(a.B);
        for (int &x : table) x = in(0, 9) ? in(0, a.pages - 1) : far[in(0, 8)];
        for (int &x : start) x = in(0, 3) ? in(-a.N, 64 * a.table_len) : far[in(0, 8)];
        for (int &x : count) x = in(0, 3) ? in(0, a.N) : far[in(0, 8)];
        a.table = table.data();
        a.start = in(0, 3) ? start.data() : nullptr;
        a.count = in(0, 1) ? count.data() : nullptr;
        std::vector<int> stored(a.B * a.N * 2 * a.Hkv);
        std::vector<char> lost(a.B);
        for (int64_t i = 0; i < 2 * (int64_t)a.B * a.Hkv * pages_of(a.N); ++i) {
            const Spot s(a, (unsigned)i);
            wrong += s.b < 0 || s.b >= a.B || s.hk < 0 || s.hk >= a.Hkv;
            wrong += s.page < -1 || s.page >= a.pages || s.lo < 0 || (s.lo < s.hi && s.hi > kPage);
            lost[s.b] |= s.lost;
            if (s.page < 0) continue;
            for (int t = s.lo; t < s.hi; ++t) {
                const int n = s.token + t;
                if (n < 0 || n >= a.N) { ++wrong; continue; }
                ++stored[((s.b * a.N + n) * a.Hkv + s.hk) * 2 + s.kind];
                const int64_t p = (a.start ? (int64_t)start[s.b] : 0) + n;
                wrong += p < 0 || p >= 64LL * a.table_len || table[s.b * a.table_sb + p / 64] != s.page || p % 64 != t;
            }
        }
        for (int b = 0; b < a.B; ++b) {
            bool any = false;
            for (int n = 0; n < a.N; ++n) {
                const int64_t p = (a.start ? (int64_t)start[b] : 0) + n;
                const bool asked = n < (a.count ? count[b] : a.N), there = p >= 0 && p < 64LL * a.table_len;
                const int entry = there ? table[b * a.table_sb + p / 64] : -1;
                const bool has = asked && there && entry >= 0 && entry < a.pages;
                any |= asked && !has;
                for (int j = 0; j < 2 * a.Hkv; ++j) wrong += stored[(b * a.N + n) * 2 * a.Hkv + j] != (has ? 1 : 0);
            }
            wrong += any != (bool)lost[b];
        }
        // the attention's walk over a sequence's pages, and its masks
        const Band w = {nullptr, a.N, 64 * a.table_len, in(1, 400), in(0, 200)};
        const int lo = in(0, 64 * a.table_len - 1), hi = in(0, 7) ? lo + in(0, 64 * a.table_len - 1 - lo) : lo - 1;
        wrong += walks<64>(w, lo, hi, 64 * a.table_len) + walks<128>(w, lo, hi, 64 * a.table_len);
        if (turn % 100 == 0) {
            const int up = least(hi, lo + in(0, 140));
            wrong += pairs<64>(w, lo, up, 64 * a.table_len) + pairs<128>(w, lo, up, 64 * a.table_len);
        }
        const int k0 = 16 * in(0, 4 * a.table_len - 1), p = in(-1, 64 * a.table_len - 1);
        for (int i = 0; i < 32; ++i) {
            wrong += (keys_of(w, p, k0) >> i & 1) != w.sees(p, k0 + i);
            bool some = false;
            for (int x = lo; x <= hi; ++x) some |= w.sees(x, k0 + i);
            wrong += some && !(keys_between(w, lo, hi, k0) >> i & 1);
            wrong += !some && lo <= hi && k0 + i > hi && (keys_between(w, lo, hi, k0) >> i & 1);
            wrong += (queries_of(w, k0, p, hi) >> i & 1) != (p + i < hi && w.sees(p + i, k0));
        }
    }
    printf("%d\n", wrong);
    return wrong != 0;
}
"""


def test_where_the_kernels_blocks_read_and_write(tmp_path):
    import os
    src, exe = tmp_path / "spots.cpp", tmp_path / "spots"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.dirname(_native.HEADER), "-I", cuda, "-o", str(exe),
                    str(src)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "0\n"


def test_the_references_8_bit_values():
    # against torch's conversion, which rounds to nearest even too, on every tie and next to it
    byte = torch.arange(256, dtype=torch.uint8)
    v = cache_ref.decode(byte)
    t = byte.view(torch.float8_e4m3fn).double()
    assert torch.equal(v.isnan(), t.isnan()) and torch.equal(v[~v.isnan()], t[~t.isnan()])
    ties = (cache_ref.VALUES[1:] + cache_ref.VALUES[:-1]) / 2
    x = torch.cat([cache_ref.VALUES, ties, ties * (1 + 2.0 ** -20), ties * (1 - 2.0 ** -20)])
    x = torch.cat([x, -x])
    assert torch.equal(cache_ref.nearest(x), x.float().to(torch.float8_e4m3fn).view(torch.uint8))
    assert int(cache_ref.nearest(torch.tensor([1e9], dtype=torch.float64))) == 126
    for top, want in ((448.0, 1.0), (449.0, 2.0), (447.0, 1.0), (1.75, 2.0 ** -8), (1.0, 2.0 ** -8), (1e-40, 2.0 ** -100),
                      (0.0, 2.0 ** -100), (3e38, 2.0 ** 120)):
        assert cache_ref.scale_of(torch.tensor([0.1 * top, -top], dtype=torch.float64)) == want, top
    assert cache_ref.scale_of(torch.tensor([math.nan, math.inf, 448.0])) == 1.0
