"""The query/key norm with the position rotation on the GPU: values and
gradients against the definition in 64 bits (tests/cross_ref.py), over head
counts, rotations, positions, strides and types."""
import ctypes
import math

import pytest
import torch

from cross_ref import check, qk_norm
from sparse_head_self_gb300 import _native, api

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _case(dtype, B, N, heads, rot, weights=(True, True), table=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x = rand(B, N, sum(heads) * 64)
    w = [(1 + 0.2 * torch.randn(64, generator=g, device="cuda")).to(dtype) if f else None for f in weights]
    rotary = api.rotary_tables(api.rotary_angles(table or N, rot, device="cuda")) if rot else None
    grads = [rand(B, h, N, 64) if h else None for h in heads]
    return x, w, rotary, grads


def _check(x, heads, w, rotary, grads, positions=None, interleaved=False, eps=1e-6):
    how = dict(eps=eps, rotary=rotary, positions=positions, interleaved=interleaved)
    out = api.qk_norm_fwd(x, heads, *w, **how)
    back = api.qk_norm_bwd(x, heads, *w, *grads, **how)
    torch.cuda.synchronize()
    want = qk_norm(x, heads, *w, eps, rotary, positions, interleaved)
    for name, t, h in zip("QKV", out, heads):
        assert (t is None) == (h == 0)
        if h:
            check(name, t, want[name])
    want = qk_norm(x, heads, *w, eps, rotary, positions, interleaved, grads)
    check("dx", back[0], want["dx"])
    for name, t, wt in (("dwq", back[1], w[0]), ("dwk", back[2], w[1])):
        assert (t is None) == (wt is None)
        if wt is not None:
            check(name, t, want[name])
    return out, back


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, (1, 1, 1)), (3, 5, (4, 2, 2)), (2, 197, (12, 12, 12)), (1, 33, (7, 3, 5)),
                                  (2, 9, (16, 0, 0)), (2, 9, (0, 4, 4)), (1, 8, (0, 0, 3)), (1, 300, (64, 1, 1))],
                         ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}")
@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (32, True), (48, False), (48, True), (64, False),
                                             (64, True)])
def test_values_and_gradients(dtype, size, rot, interleaved):
    B, N, heads = size
    x, w, rotary, grads = _case(dtype, B, N, heads, rot)
    _check(x, heads, w, rotary, grads, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("weights", [(False, False), (True, False), (False, True)])
def test_without_one_norm_or_both(dtype, weights):
    x, w, rotary, grads = _case(dtype, 2, 21, (4, 3, 2), 32, weights)
    _check(x, (4, 3, 2), w, rotary, grads)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_positions(dtype, interleaved):
    x, w, rotary, grads = _case(dtype, 3, 11, (4, 2, 2), 64, table=5000)
    g = torch.Generator(device="cuda").manual_seed(1)
    each = torch.randint(-1, 5000, (3, 11), generator=g, device="cuda", dtype=torch.int32)
    one = torch.arange(11, device="cuda", dtype=torch.int32) - 1        # a class token first
    wide = torch.randint(-1, 5000, (3, 17), generator=g, device="cuda", dtype=torch.int32)[:, 3:14]
    for p in (each, one, wide, one[None].expand(3, 11)):
        out, _ = _check(x, (4, 2, 2), w, rotary, grads, p, interleaved)
    # a token at a negative position is not rotated: as in a call where none is (which _check
    # compares with the norm alone)
    off = torch.full((11,), -1, dtype=torch.int32, device="cuda")
    none, _ = _check(x, (4, 2, 2), w, rotary, grads, off, interleaved)
    assert torch.equal(out[0][:, :, 0], none[0][:, :, 0])


def test_position_behind_the_table_is_reported():
    x, w, rotary, grads = _case(BF16, 1, 6, (2, 2, 2), 64)
    pos = torch.tensor([0, 1, 6, 2, 2**31 - 1, 5], dtype=torch.int32, device="cuda")
    _check(x, (2, 2, 2), w, rotary, grads, pos)                         # those two are not rotated
    code = ctypes.c_uint(0)
    _native.check(_native.lib().fibatt_device_error(1, ctypes.byref(code)))
    assert code.value == 8
    _native.check(_native.lib().fibatt_device_error(1, ctypes.byref(code)))
    assert code.value == 0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_strided_tokens(dtype):
    x, w, rotary, grads = _case(dtype, 3, 14, (3, 2, 2), 64)
    big = torch.full((3, 20, 7 * 64 + 24), math.nan, dtype=dtype, device="cuda")
    view = big[:, 4:18, 8:8 + 7 * 64]
    view.copy_(x)
    a = api.qk_norm_fwd(x, (3, 2, 2), *w, rotary=rotary)
    b = api.qk_norm_fwd(view, (3, 2, 2), *w, rotary=rotary)
    c = api.qk_norm_fwd(x[:1].expand(3, -1, -1), (3, 2, 2), *w, rotary=rotary)
    for i, j, k in zip(a, b, c):
        assert torch.equal(i, j) and torch.equal(k, i[:1].expand_as(k))
    for i, j in zip(api.qk_norm_bwd(x, (3, 2, 2), *w, *grads, rotary=rotary),
                    api.qk_norm_bwd(view, (3, 2, 2), *w, *grads, rotary=rotary)):
        assert torch.equal(i, j)


def test_extreme_rows():
    # rows of zeros, of one large value, near the smallest and the largest of the type
    x, w, rotary, grads = _case(F32, 1, 6, (2, 2, 1), 64)
    x[0, 0] = 0
    x[0, 1] = 0
    x[0, 1, ::64] = 1e15
    x[0, 2] *= 1e-18
    x[0, 3] *= 1e17
    _check(x, (2, 2, 1), w, rotary, grads, eps=1e-6)
    # a NaN stays in its own head and in its own weight's gradient
    x, w, rotary, grads = _case(BF16, 1, 6, (2, 2, 2), 64)
    ref = api.qk_norm_bwd(x, (2, 2, 2), *w, *grads, rotary=rotary)
    x[0, 3, 70] = math.nan                       # a query head
    grads[2][0, 1, 2, 5] = math.nan              # a value head's gradient
    dx, dwq, dwk = api.qk_norm_bwd(x, (2, 2, 2), *w, *grads, rotary=rotary, eps=0.0)
    assert bool(torch.isnan(dwq).any()) and not bool(torch.isnan(dwk).any())
    bad = torch.isnan(dx).view(6, 6, 64).any(-1)
    assert {tuple(map(int, i)) for i in bad.nonzero()} == {(3, 1), (2, 5)}
    assert ref[0].shape == dx.shape


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_differences(dtype):
    # the gradient along a direction against the definition's differences in 64 bits
    x, w, rotary, grads = _case(dtype, 2, 7, (3, 2, 2), 32)
    back = api.qk_norm_bwd(x, (3, 2, 2), *w, *grads, rotary=rotary)
    want = qk_norm(x, (3, 2, 2), *w, 1e-6, rotary, None, False, grads)

    def loss(xx, wq, wk):
        out = qk_norm(xx, (3, 2, 2), wq, wk, 1e-6, rotary)
        return sum(float((out[n][0] * g.double()).sum()) for n, g in zip("QKV", grads))

    g = torch.Generator(device="cuda").manual_seed(5)
    args = [x.double(), w[0].double(), w[1].double()]
    for i, (name, got) in enumerate(zip(("dx", "dwq", "dwk"), back)):
        d = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(args), list(args)
        h = 1e-5
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        diff = (loss(*up) - loss(*down)) / (2 * h)
        bound = float((want[name][1] * d.abs()).sum())
        # the differences' own error: h^2 of third derivatives and 2^-53 / h of the loss
        assert abs(float((got.double() * d).sum()) - diff) <= bound + 1e-5 * (1 + abs(diff)), name


def test_repeat_streams_and_graphs():
    heads = (12, 4, 4)
    x, w, rotary, grads = _case(BF16, 8, 197, heads, 64)
    first = api.qk_norm_fwd(x, heads, *w, rotary=rotary) + api.qk_norm_bwd(x, heads, *w, *grads, rotary=rotary)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = []
    for _ in range(3):
        for s in streams:
            out.append(api.qk_norm_fwd(x, heads, *w, rotary=rotary, stream=s)
                       + api.qk_norm_bwd(x, heads, *w, *grads, rotary=rotary, stream=s))
    torch.cuda.synchronize()
    for o in out:
        assert all(torch.equal(a, b) for a, b in zip(first, o))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = api.qk_norm_fwd(x, heads, *w, rotary=rotary) + api.qk_norm_bwd(x, heads, *w, *grads, rotary=rotary)
    x.copy_(_case(BF16, 8, 197, heads, 64, seed=9)[0])
    graph.replay()
    torch.cuda.synchronize()
    want = api.qk_norm_fwd(x, heads, *w, rotary=rotary) + api.qk_norm_bwd(x, heads, *w, *grads, rotary=rotary)
    assert all(torch.equal(a, b) for a, b in zip(want, o))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_autograd(dtype):
    heads = (4, 2, 2)
    x, w, rotary, grads = _case(dtype, 2, 13, heads, 64)
    x.requires_grad_()
    wq, wk = (t.requires_grad_() for t in w)
    q, k, v = api.qk_norm(x, heads, wq, wk, rotary=rotary)
    torch.autograd.backward([q, k, v], grads)
    want = qk_norm(x.detach(), heads, wq.detach(), wk.detach(), 1e-6, rotary, None, False, grads)
    check("dx", x.grad, want["dx"])
    check("dwq", wq.grad, want["dwq"])
    check("dwk", wk.grad, want["dwk"])
    # only the keys are used: the others' gradients are zeros
    x.grad = None
    api.qk_norm(x, heads, wq.detach(), wk.detach(), rotary=rotary)[1].backward(grads[1])
    zero = [torch.zeros_like(grads[0]), grads[1], torch.zeros_like(grads[2])]
    check("dx", x.grad, qk_norm(x.detach(), heads, wq.detach(), wk.detach(), 1e-6, rotary, None, False, zero)["dx"])


def test_autograd_of_inputs_that_have_to_be_copied():
    heads = (2, 1, 1)
    g = torch.Generator(device="cuda").manual_seed(6)
    base = torch.randn(2, 9, 4 * 64 + 1, generator=g, device="cuda", requires_grad=True)
    grads = [torch.randn(2, h, 9, 64, generator=g, device="cuda") for h in heads]
    x = base[..., 1:]                       # tokens off 16 bytes
    torch.autograd.backward(list(api.qk_norm(x, heads)), grads)
    want = qk_norm(x.detach(), heads, None, None, 1e-6, None, None, False, grads)
    check("dx", base.grad[..., 1:], want["dx"])
    y = torch.randn(1, 1, 4 * 64, generator=g, device="cuda", requires_grad=True)    # one token everywhere
    torch.autograd.backward(list(api.qk_norm(y.expand(2, 9, -1), heads)), grads)
    value, bound = qk_norm(y.detach().expand(2, 9, -1), heads, None, None, 1e-6, None, None, False, grads)["dx"]
    # autograd's sum of eighteen: as many roundings of the largest partial sum
    check("dx", y.grad, (value.sum((0, 1), keepdim=True), (bound + 18 * 2.0 ** -24 * value.abs()).sum((0, 1), keepdim=True)))


def test_gpu_refusals():
    x, w, rotary, grads = _case(BF16, 2, 5, (2, 1, 1), 64)
    with pytest.raises(ValueError, match="values a token"):
        api.qk_norm_fwd(x, (2, 2, 1), *w)
    with pytest.raises(ValueError, match="q_weight"):
        api.qk_norm_fwd(x, (2, 1, 1), w[0].float(), w[1])
    with pytest.raises(ValueError, match="positions"):
        api.qk_norm_fwd(x, (2, 1, 1), *w, positions=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="positions"):
        api.qk_norm_fwd(x, (2, 1, 1), *w, rotary=rotary, positions=torch.zeros(5, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="sin"):
        api.qk_norm_fwd(x, (2, 1, 1), *w, rotary=(rotary[0], rotary[1][:3]))
    with pytest.raises(api.FibattError, match="tables of 3 positions"):
        api.qk_norm_fwd(x, (2, 1, 1), *w, rotary=tuple(t[:3].contiguous() for t in rotary))
    with pytest.raises(ValueError, match="dK"):
        api.qk_norm_bwd(x, (2, 1, 1), *w, grads[0], grads[0], grads[2])
    with pytest.raises(api.FibattError, match="workspace"):
        api.qk_norm_bwd(x, (2, 1, 1), *w, *grads, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_what_the_backward_reads_may_not_change_before_it():
    x, w, rotary, _ = _case(BF16, 2, 5, (2, 1, 1), 64)
    x = x.detach().requires_grad_()
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    q, _, _ = api.qk_norm(x, (2, 1, 1), *w, rotary=tuple(t.clone() for t in rotary), positions=pos)
    pos -= 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        q.sum().backward()


def test_workspaces_of_other_places_are_refused():
    x, w, _, grads = _case(BF16, 2, 5, (2, 1, 1), 64)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        api.qk_norm_bwd(x, (2, 1, 1), *w, *grads, workspace=torch.empty(1 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_gradients_weights_and_tables_off_16_bytes(dtype):
    # contiguous parts of larger tensors: a gradient through a concatenation behind one element,
    # weights and tables in a flat buffer behind one
    heads = (4, 2, 2)
    x, w, rotary, grads = _case(dtype, 2, 13, heads, 64)
    x.requires_grad_()
    flat = torch.cat([w[0][:1], *w]).requires_grad_()
    wide = [torch.cat([t.flatten()[:1], t.flatten()])[1:].view_as(t) for t in rotary]
    assert flat[1:].data_ptr() % 16 and all(t.is_contiguous() and t.data_ptr() % 16 for t in wide)
    out = api.qk_norm(x, heads, flat[1:65], flat[65:], rotary=wide)
    joined = torch.cat([t for o in out for t in (x.new_zeros(1), o.flatten())])
    joined.backward(torch.cat([t for g in grads for t in (x.new_zeros(1), g.flatten())]))
    want = qk_norm(x.detach(), heads, *w, 1e-6, rotary, None, False)
    for name, t in zip("QKV", out):
        check(name, t.detach(), want[name])
    want = qk_norm(x.detach(), heads, *w, 1e-6, rotary, None, False, grads)
    check("dx", x.grad, want["dx"])
    check("dwq", flat.grad[1:65], want["dwq"])
    check("dwk", flat.grad[65:], want["dwk"])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("weights", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_gradient_without_a_norm_does_not_depend_on_the_input(dtype, weights, bad):
    heads = (4, 3, 2)
    x, w, rotary, grads = _case(dtype, 2, 21, heads, 32, weights)
    want = api.qk_norm_bwd(x, heads, *w, *grads, rotary=rotary)
    h = x.view(2, 21, 9, 64)
    if not weights[0]:
        h[:, 3::5, :4, 7] = bad
    if not weights[1]:
        h[:, ::4, 4:7, 50] = bad
    h[:, :, 7:] = bad                # values: copied, whatever they are
    got = api.qk_norm_bwd(x, heads, *w, *grads, rotary=rotary)
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    # large finite gradients and inputs, whose product is beyond the type: dx is dy turned back
    if not any(weights):
        big = [g * 1e30 for g in grads]
        ref = qk_norm(torch.zeros_like(x), heads, None, None, 1e-6, rotary, None, False, big)["dx"]
        check("dx", api.qk_norm_bwd(torch.full_like(x, 1e30), heads, None, None, *big, rotary=rotary)[0], ref)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 32, 64])
def test_what_is_not_rotated_keeps_its_infinities(dtype, interleaved, rot):
    # dims behind rot_dims, and tokens at a negative position: copied when there is no norm, in both directions
    heads = (3, 2, 1)
    x, _, rotary, grads = _case(dtype, 2, 19, heads, rot)
    pos = torch.arange(19, device="cuda", dtype=torch.int32) - 1        # a class token first
    pos[7] = -5
    off = pos < 0
    h = x.view(2, 19, 6, 64)
    for t in (h.transpose(1, 2), *grads):      # [B, H, N, 64]
        t[:, :, off, 3::9] = math.inf
        t[:, :, off, 5::11] = -math.inf
        if rot < 64:
            t[:, :, 2::5, rot::7] = math.inf
            t[:, :, 2::5, rot + 1::7] = math.nan
    how = dict(rotary=rotary, positions=pos, interleaved=interleaved)
    out = api.qk_norm_fwd(x, heads, **how)
    dx = api.qk_norm_bwd(x, heads, None, None, *grads, **how)[0].view(2, 19, 6, 64).transpose(1, 2)
    first = 0
    for i, n in enumerate(heads):
        for got, src in ((out[i], h.transpose(1, 2)[:, first:first + n]), (dx[:, first:first + n], grads[i])):
            kept = torch.ones_like(got, dtype=torch.bool)
            if i < 2:                          # value heads are copied altogether
                kept[:, :, ~off, :rot] = False
            assert torch.equal(got[kept].nan_to_num(7.0, 9e9, -9e9), src[kept].nan_to_num(7.0, 9e9, -9e9))
            assert bool(got[~kept].isfinite().all())
        first += n


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,N", [(1, 9), (3, 1), (1, 1)])
def test_strides_of_one_sequence_or_one_token_do_not_matter(dtype, B, N):
    heads = (2, 1, 1)
    x, w, rotary, grads = _case(dtype, B, N, heads, 64)
    C = 4 * 64
    odd = torch.as_strided(x, (B, N, C), (N * C if B > 1 else N * C + 1, C if N > 1 else C + 3, 1))
    assert torch.equal(odd, x) and odd.stride() != x.stride()
    for a, b in zip(api.qk_norm_fwd(x, heads, *w, rotary=rotary) + api.qk_norm_bwd(x, heads, *w, *grads, rotary=rotary),
                    api.qk_norm_fwd(odd, heads, *w, rotary=rotary) + api.qk_norm_bwd(odd, heads, *w, *grads, rotary=rotary)):
        assert torch.equal(a, b)
    odd.requires_grad_()
    torch.autograd.backward(list(api.qk_norm(odd, heads, *w, rotary=rotary)), grads)
    check("dx", odd.grad, qk_norm(x, heads, *w, 1e-6, rotary, None, False, grads)["dx"])


@pytest.mark.parametrize("B,N,heads,interleaved", [(2, 16385, (16, 16, 0), False), (256, 197, (12, 12, 0), False),
                                                   (1, 6000, (7, 3, 2), True)])
def test_weights_gradients_keep_their_digits_over_many_rows(B, N, heads, interleaved):
    # In the mean square a rounding to 32 bits is 2^-24 / sqrt(3) of its value at most.  A term of dw
    # has about 8 (its rotation 3, x r and r 4, its product 1); a lane adds the terms of a unit, n
    # at most, whose partial sums add sqrt(n / 2) of a rounding; then two joins of lanes, and one
    # rounding each of a warp's, a block's and the result's value.  No count grows with the rows.
    x, w, rotary, _ = _case(F32, B, N, heads, 64)
    g = torch.Generator(device="cuda").manual_seed(8)
    grads = [torch.randn(B, h, N, 64, generator=g, device="cuda") if h else None for h in heads]
    got = api.qk_norm_bwd(x, heads, *w, *grads, rotary=rotary, interleaved=interleaved)[1:]
    want = [0.0, 0.0]
    for lo in range(0, B, 64):
        at = slice(lo, lo + 64)
        part = qk_norm(x[at], heads, *w, 1e-6, rotary, None, interleaved, [None if t is None else t[at] for t in grads])
        want = [a + part[n][0] for a, n in zip(want, ("dwq", "dwk"))]
    for i, h in enumerate(heads[:2]):
        n = 2 * -(-h // 4) if h > 4 else 2
        bound = 2.0 ** -24 / math.sqrt(3) * math.sqrt(8 + n / 2 + 2 + 3)
        err = float((got[i].double() - want[i]).norm() / want[i].norm())
        assert err <= bound, (i, err, bound)


def test_weights_gradients_that_overflow_are_infinite():
    x, w, _, grads = _case(F32, 4, 200, (4, 4, 1), 0)
    grads[0][..., 5] = 3e38 * x.view(4, 200, 9, 64)[:, :, :4, 5].transpose(1, 2).sign()
    _, dwq, dwk = api.qk_norm_bwd(x, (4, 4, 1), *w, *grads)
    assert float(dwq[5]) == math.inf and bool(dwq[:5].isfinite().all()) and bool(dwq[6:].isfinite().all())
    assert bool(dwk.isfinite().all())
