"""Python binding of libfibatt: same names as the C ABI, argument marshalling only.

Every step of the attention runs in the library's CUDA kernels; torch is used
for device memory, dtypes and the current stream.  There is no CPU fallback:
calls on CPU tensors are rejected.
"""
from __future__ import annotations

import ctypes
import operator
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _native
from ._native import FibattError, check, lib

HEAD_DIM = 64

_DTYPES = {torch.float32: _native.F32, torch.bfloat16: _native.BF16}
_WEIGHT_SHAPE = (HEAD_DIM,)


# ------------------------------------------------------------------ helpers

def wythoff_row(i: int) -> tuple[int, int]:
    """(a_i, b_i) of Wythoff row i (Fibottention Sec. 3.2)."""
    a, b = ctypes.c_int64(), ctypes.c_int64()
    check(lib().fibatt_wythoff_row(int(i), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def wythoff_row_modified(i: int) -> tuple[int, int]:
    """The two terms preceding Wythoff row i (README Algorithm 2, modified variant)."""
    a, b = ctypes.c_int64(), ctypes.c_int64()
    check(lib().fibatt_wythoff_row_modified(int(i), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def window_schedule(h: int, w_min: int, w_max: int) -> list[int]:
    """Per-head windows w_1..w_h (Fibottention Sec. 3.2)."""
    w = (ctypes.c_int64 * h)()
    check(lib().fibatt_window_schedule(int(h), int(w_min), int(w_max), w))
    return list(w)


def _i64(xs):
    xs = [int(x) for x in xs]
    return (ctypes.c_int64 * max(1, len(xs)))(*xs)


def _i32(xs):
    xs = [int(x) for x in xs]
    return (ctypes.c_int32 * max(1, len(xs)))(*xs)


class Support:
    """Owner of a ``fibatt_support_t`` handle (host memory only)."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle
        H, N, total = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        check(lib().fibatt_support_info(self._h, ctypes.byref(H), ctypes.byref(N), ctypes.byref(total)))
        self.H, self.N, self.total_entries = H.value, N.value, total.value

    # -- constructors --------------------------------------------------------
    @classmethod
    def build(cls, N: int, a, b, w, include_diag: bool) -> "Support":
        """fibatt_support_build: head h uses Fib(a[h], b[h]) within window w[h]."""
        H = len(a)
        assert len(b) == H and len(w) == H
        h = ctypes.c_void_p()
        check(lib().fibatt_support_build(H, int(N), _i64(a), _i64(b), _i64(w), int(bool(include_diag)),
                                         ctypes.byref(h)))
        return cls(h)

    @classmethod
    def from_distances(cls, N: int, distances: list, include_diag: bool) -> "Support":
        """fibatt_support_build_distances: head h attends |j-k| in distances[h]."""
        counts = [len(d) for d in distances]
        flat = [int(x) for d in distances for x in d]
        h = ctypes.c_void_p()
        check(lib().fibatt_support_build_distances(len(distances), int(N), _i32(counts), _i32(flat),
                                                   int(bool(include_diag)), ctypes.byref(h)))
        return cls(h)

    @classmethod
    def wythoff(cls, H: int, N: int, w_min: int, w_max: int, include_diag: bool,
                modified: bool = False, permutation=None) -> "Support":
        """Fibottention's layer support: head i on Wythoff row pi(i) (rows 1..H),
        windows from the linear schedule."""
        row = wythoff_row_modified if modified else wythoff_row
        ab = [row(i) for i in range(1, H + 1)]
        w = window_schedule(H, w_min, w_max)
        perm = list(range(H)) if permutation is None else [int(p) for p in permutation]
        assert sorted(perm) == list(range(H))
        return cls.build(N, [ab[p][0] for p in perm], [ab[p][1] for p in perm], [w[p] for p in perm],
                         include_diag)

    def set_global_token(self, enabled: bool = True) -> "Support":
        """fibatt_support_set_global_token: token 0 attends every key and is
        attended by every query (README Algorithm 2's class token)."""
        check(lib().fibatt_support_set_global_token(self._h, int(bool(enabled))))
        return self

    # -- queries -------------------------------------------------------------
    def tables(self):
        """(counts[H], signed offsets (CSR), pairs[H])."""
        counts = (ctypes.c_int32 * self.H)()
        offs = (ctypes.c_int32 * max(1, self.total_entries))()
        pairs = (ctypes.c_int64 * self.H)()
        check(lib().fibatt_support_get(self._h, counts, offs, pairs))
        return list(counts), list(offs)[: self.total_entries], list(pairs)

    def head_offsets(self) -> list[list[int]]:
        counts, offs, _ = self.tables()
        out, p = [], 0
        for c in counts:
            out.append(offs[p:p + c])
            p += c
        return out

    @property
    def pairs(self) -> list[int]:
        return self.tables()[2]

    def total_pairs(self, B: int = 1) -> int:
        return B * sum(self.pairs)

    def bwd_workspace_bytes(self, B: int) -> int:
        return int(lib().fibatt_bwd_workspace_bytes(self._h, int(B)))

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().fibatt_support_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------------- attention

def _check_io(name: str, t: torch.Tensor, shape, dtype, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (libfibatt has no CPU path)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream_ptr(stream, device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def fwd(support: Support, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, scale: float,
        O: torch.Tensor | None = None, LSE: torch.Tensor | None = None, stream=None):
    """fibatt_fwd on [B, H, N, 64] CUDA tensors; returns (O, LSE)."""
    if Q.dim() != 4:
        raise ValueError("Q must be [B, H, N, D]")
    B, H, N, D = Q.shape
    if (H, N) != (support.H, support.N):
        raise ValueError(f"tensors have H={H}, N={N}; support has H={support.H}, N={support.N}")
    if Q.dtype not in _DTYPES:
        raise ValueError(f"dtype {Q.dtype} unsupported (float32 or bfloat16)")
    dev = Q.device
    for n, t in (("Q", Q), ("K", K), ("V", V)):
        _check_io(n, t, Q.shape, Q.dtype, dev)
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None:
        LSE = torch.empty((B, H, N), dtype=torch.float32, device=dev)
    _check_io("O", O, Q.shape, Q.dtype, dev)
    _check_io("LSE", LSE, (B, H, N), torch.float32, dev)
    check(lib().fibatt_fwd(support.handle, B, D, _DTYPES[Q.dtype], Q.data_ptr(), K.data_ptr(),
                           V.data_ptr(), float(scale), O.data_ptr(), LSE.data_ptr(),
                           _stream_ptr(stream, dev)))
    return O, LSE


def bwd(support: Support, Q, K, V, O, LSE, dO, scale: float, dQ=None, dK=None, dV=None,
        workspace: torch.Tensor | None = None, stream=None):
    """fibatt_bwd on [B, H, N, 64] CUDA tensors; returns (dQ, dK, dV)."""
    B, H, N, D = Q.shape
    if (H, N) != (support.H, support.N):
        raise ValueError(f"tensors have H={H}, N={N}; support has H={support.H}, N={support.N}")
    if Q.dtype not in _DTYPES:
        raise ValueError(f"dtype {Q.dtype} unsupported (float32 or bfloat16)")
    dev = Q.device
    for n, t in (("Q", Q), ("K", K), ("V", V), ("O", O), ("dO", dO)):
        _check_io(n, t, Q.shape, Q.dtype, dev)
    _check_io("LSE", LSE, (B, H, N), torch.float32, dev)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(Q) if dK is None else dK
    dV = torch.empty_like(Q) if dV is None else dV
    for n, t in (("dQ", dQ), ("dK", dK), ("dV", dV)):
        _check_io(n, t, Q.shape, Q.dtype, dev)
    need = support.bwd_workspace_bytes(B)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check(lib().fibatt_bwd(support.handle, B, D, _DTYPES[Q.dtype], Q.data_ptr(), K.data_ptr(),
                           V.data_ptr(), O.data_ptr(), LSE.data_ptr(), dO.data_ptr(), float(scale),
                           dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), ws_ptr, ws_bytes,
                           _stream_ptr(stream, dev)))
    return dQ, dK, dV


def bwd_noalloc(support: Support, Q, K, V, O, LSE, dO, scale: float, dQ, dK, dV, stream=None):
    """fibatt_bwd_noalloc: the backward pass without any workspace argument, for
    callers that must not allocate device memory (its scratch is a fixed array
    inside the library; at most B*H*N = FIBATT_NOALLOC_MAX_ROWS rows).  The
    output tensors dQ, dK, dV are required and written in place."""
    B, H, N, D = Q.shape
    if (H, N) != (support.H, support.N):
        raise ValueError(f"tensors have H={H}, N={N}; support has H={support.H}, N={support.N}")
    if Q.dtype not in _DTYPES:
        raise ValueError(f"dtype {Q.dtype} unsupported (float32 or bfloat16)")
    dev = Q.device
    for n, t in (("Q", Q), ("K", K), ("V", V), ("O", O), ("dO", dO), ("dQ", dQ), ("dK", dK), ("dV", dV)):
        _check_io(n, t, Q.shape, Q.dtype, dev)
    _check_io("LSE", LSE, (B, H, N), torch.float32, dev)
    check(lib().fibatt_bwd_noalloc(support.handle, B, D, _DTYPES[Q.dtype], Q.data_ptr(), K.data_ptr(),
                                   V.data_ptr(), O.data_ptr(), LSE.data_ptr(), dO.data_ptr(), float(scale),
                                   dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), _stream_ptr(stream, dev)))
    return dQ, dK, dV


class FibottentionFunction(torch.autograd.Function):
    """Autograd wrapper: forward = fibatt_fwd, backward = fibatt_bwd."""

    @staticmethod
    def forward(ctx, Q, K, V, support: Support, scale: float):
        Q, K, V = Q.contiguous(), K.contiguous(), V.contiguous()
        O, LSE = fwd(support, Q, K, V, scale)
        ctx.save_for_backward(Q, K, V, O, LSE)
        ctx.support = support
        ctx.scale = scale
        return O

    @staticmethod
    def backward(ctx, dO):
        Q, K, V, O, LSE = ctx.saved_tensors
        dQ, dK, dV = bwd(ctx.support, Q, K, V, O, LSE, dO.contiguous(), ctx.scale)
        return dQ, dK, dV, None, None


def fibottention(Q, K, V, support: Support, scale: float | None = None):
    """Differentiable Fibottention attention on [B, H, N, 64] CUDA tensors."""
    if scale is None:
        scale = Q.shape[-1] ** -0.5
    return FibottentionFunction.apply(Q, K, V, support, float(scale))


# ---------------------------------------------------- query and key norms

def _check_tensor(name: str, t, dtype, index: int) -> None:
    """A CUDA tensor of this type on device `index`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libfibatt has no CPU path)")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _check_dense(name: str, t, shape, dtype, index: int) -> int:
    """The address of a contiguous tensor of this shape."""
    _check_tensor(name, t, dtype, index)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _index(name: str, t) -> int:
    """The device index of a CUDA tensor."""
    index = t.get_device()
    if index < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libfibatt has no CPU path)")
    return index


def _workspace(ws, need: int, index: int):
    """The caller's scratch memory, or fresh memory of `need` bytes."""
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=f"cuda:{index}")
    _check_dense("workspace", ws, ws.shape if isinstance(ws, torch.Tensor) else None, getattr(ws, "dtype", None), index)
    return ws


_device_of_thread = torch._C._cuda_getDevice
_stream_of_thread = torch._C._cuda_getCurrentRawStream


def _launch(index: int, stream, call, *args):
    """call(*args, stream pointer) with the launching stream and its device
    current: what a call allocates then belongs to the stream that uses it."""
    if stream is not None:
        if stream.device_index != index:
            raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{index}")
        with torch.cuda.stream(stream):
            return call(*args, stream.cuda_stream)
    if index != _device_of_thread():
        with torch.cuda.device(index):
            return call(*args, _stream_of_thread(index))
    return call(*args, _stream_of_thread(index))


def rotary_tables(angles: torch.Tensor):
    """(cos, sin) for qk_norm from a table of angles [positions, pairs] (any
    float type; far positions want float64): fp32, contiguous."""
    if angles.dim() != 2 or angles.shape[1] not in (8, 16, 24, 32):
        raise ValueError("angles must be [positions, pairs] with 8, 16, 24 or 32 pairs")
    return angles.cos().float().contiguous(), angles.sin().float().contiguous()


def rotary_angles(positions: int, rot_dims: int = HEAD_DIM, theta: float = 10000.0, device=None) -> torch.Tensor:
    """Angles p theta^(-2 i / rot_dims) of positions 0..positions - 1, float64."""
    half = rot_dims // 2
    freq = theta ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    return torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq


def rotary_angles_2d(height: int, width: int, rot_dims: int = HEAD_DIM, theta: float = 100.0,
                     device=None) -> torch.Tensor:
    """Angles of a height x width grid of patches, row by row: the first half
    of the pairs turns with the patch's row, the second with its column."""
    if rot_dims % 4:
        raise ValueError("rot_dims must be a multiple of 4")
    rows = rotary_angles(height, rot_dims // 2, theta, device)
    cols = rotary_angles(width, rot_dims // 2, theta, device)
    return torch.cat([rows[:, None].expand(-1, width, -1), cols[None].expand(height, -1, -1)], -1).reshape(
        height * width, rot_dims // 2)


def _norm_desc(x, heads, q_weight, k_weight, eps, rotary, positions, interleaved):
    """(packed fibatt_qk_norm, device index, B, N, Hq, Hk, Hv, x's strides)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [B, N, (Hq + Hk + Hv) * 64] tensor")
    dtype = x.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"dtype {dtype} unsupported (float32 or bfloat16)")
    index = _index("x", x)
    Hq, Hk, Hv = heads
    B, N, C = x.shape
    if min(Hq, Hk, Hv) < 0 or C != (Hq + Hk + Hv) * HEAD_DIM:
        raise ValueError(f"x has {C} values a token, heads {(Hq, Hk, Hv)} of {HEAD_DIM} need {(Hq + Hk + Hv) * HEAD_DIM}")
    sb, sn, sc = x.stride()
    if sc != 1:
        raise ValueError("x must have contiguous tokens")
    # a dim of one element has no stride that matters
    if B == 1:
        sb = 0
    if N == 1:
        sn = 0
    wq = wk = cos_ptr = sin_ptr = rot = table = pos = pos_sb = 0
    if q_weight is not None:
        wq = _check_dense("q_weight", q_weight, _WEIGHT_SHAPE, dtype, index)
    if k_weight is not None:
        wk = _check_dense("k_weight", k_weight, _WEIGHT_SHAPE, dtype, index)
    if rotary is not None:
        cos, sin = rotary
        shape = cos.shape
        cos_ptr = _check_dense("cos", cos, shape, torch.float32, index)
        sin_ptr = _check_dense("sin", sin, shape, torch.float32, index)
        if len(shape) != 2:
            raise ValueError("cos and sin must be [positions, rot_dims / 2]")
        table, rot = shape
        rot *= 2
        if positions is not None:
            _check_tensor("positions", positions, torch.int32, index)
            shape, strides = positions.shape, positions.stride()
            if (shape != (N,) and shape != (B, N)) or (N > 1 and strides[-1] != 1):
                raise ValueError(f"positions must be [N] or [B, N] with contiguous rows, got {tuple(shape)}")
            pos = positions.data_ptr()
            pos_sb = strides[0] if len(shape) == 2 else 0
    elif positions is not None:
        raise ValueError("positions without rotary tables")
    d = _native.QK_NORM.pack(B, N, Hq, Hk, Hv, HEAD_DIM, code, wq, wk, eps, rot, 1 if interleaved else 0, cos_ptr,
                             sin_ptr, table, pos, pos_sb)
    return d, index, B, N, Hq, Hk, Hv, sb, sn


def qk_norm_fwd(x: torch.Tensor, heads, q_weight=None, k_weight=None, eps: float = 1e-6, rotary=None, positions=None,
                interleaved: bool = False, stream=None):
    """fibatt_qk_norm_fwd on a packed projection x [B, N, (Hq + Hk + Hv) * 64]
    with heads = (Hq, Hk, Hv); returns (Q, K, V), [B, H, N, 64] each, None for
    a kind without heads.  rotary = (cos, sin), [positions, rot_dims / 2] fp32;
    positions int32 [N] or [B, N]."""
    d, index, B, N, Hq, Hk, Hv, sb, sn = _norm_desc(x, heads, q_weight, k_weight, eps, rotary, positions, interleaved)

    return _launch(index, stream, _qk_norm_fwd, d, x, x.dtype, x.device, B, N, Hq, Hk, Hv, sb, sn)


def _qk_norm_fwd(d, x, dtype, device, B, N, Hq, Hk, Hv, sb, sn, s):
    q = k = v = qp = kp = vp = None
    if Hq:
        q = torch.empty((B, Hq, N, HEAD_DIM), dtype=dtype, device=device)
        qp = q.data_ptr()
    if Hk:
        k = torch.empty((B, Hk, N, HEAD_DIM), dtype=dtype, device=device)
        kp = k.data_ptr()
    if Hv == Hk and Hk:
        v = torch.empty_like(k)
        vp = v.data_ptr()
    elif Hv:
        v = torch.empty((B, Hv, N, HEAD_DIM), dtype=dtype, device=device)
        vp = v.data_ptr()
    status = lib().fibatt_qk_norm_fwd(d, x.data_ptr(), sb, sn, qp, kp, vp, s)
    if status:
        check(status)
    return q, k, v


def qk_norm_bwd(x: torch.Tensor, heads, q_weight, k_weight, dQ, dK, dV, eps: float = 1e-6, rotary=None,
                positions=None, interleaved: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """fibatt_qk_norm_bwd: from the gradients of qk_norm_fwd's results (None
    for a kind without heads) to (dx, dq_weight, dk_weight); a weight that is
    None has the gradient None."""
    d, index, B, N, Hq, Hk, Hv, sb, sn = _norm_desc(x, heads, q_weight, k_weight, eps, rotary, positions, interleaved)
    grads = []
    for name, g, h in (("dQ", dQ, Hq), ("dK", dK, Hk), ("dV", dV, Hv)):
        if h:
            grads.append(_check_dense(name, g, (B, h, N, HEAD_DIM), x.dtype, index))
        else:
            grads.append(None)

    def call(s):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dqw = None if q_weight is None else torch.empty_like(q_weight)
        dkw = None if k_weight is None else torch.empty_like(k_weight)
        ws = _workspace(workspace, lib().fibatt_qk_norm_bwd_workspace_bytes(), index)
        check(lib().fibatt_qk_norm_bwd(d, x.data_ptr(), sb, sn, *grads, dx.data_ptr(), dx.stride(0), dx.stride(1),
                                       None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(),
                                       ws.data_ptr(), ws.numel() * ws.element_size(), s))
        return dx, dqw, dkw

    return _launch(index, stream, call)


def _readable(t):
    """t, or a copy that the library reads: contiguous rows, strides and start
    on 16 bytes, and (the dim before the last) no row repeated."""
    step = 16 // t.element_size()
    strides, shape = t.stride(), t.shape
    ok = (strides[-1] == 1 and t.data_ptr() % 16 == 0 and (strides[-2] > 0 or shape[-2] == 1)
          and all(s % step == 0 for s, n in zip(strides[:-1], shape) if n > 1))
    return t if ok else t.clone(memory_format=torch.contiguous_format)


def _dense(t):
    """t (or None), or a copy: contiguous and on 16 bytes, which a contiguous
    part of a larger tensor need not be (a weight in a flat buffer of all
    parameters, a gradient that comes through a concatenation)."""
    if t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class QkNormFunction(torch.autograd.Function):
    """Autograd wrapper: forward = fibatt_qk_norm_fwd, backward = fibatt_qk_norm_bwd."""

    @staticmethod
    def forward(ctx, x, q_weight, k_weight, heads, eps, rotary, positions, interleaved):
        x, q_weight, k_weight = _readable(x), _dense(q_weight), _dense(k_weight)
        ctx.how = (tuple(heads), float(eps), bool(interleaved))
        cos, sin = (None, None) if rotary is None else (_dense(t) for t in rotary)
        rotary = None if rotary is None else (cos, sin)
        ctx.save_for_backward(x, q_weight, k_weight, cos, sin, positions)
        ctx.set_materialize_grads(False)
        out = qk_norm_fwd(x, heads, q_weight, k_weight, eps, rotary, positions, interleaved)
        ctx.shapes = [None if t is None else t.shape for t in out]
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        x, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        heads, eps, interleaved = ctx.how
        rotary = None if cos is None else (cos, sin)
        grads = [g if s is None else torch.zeros(s, dtype=x.dtype, device=x.device) if g is None else _dense(g)
                 for g, s in zip(grads, ctx.shapes)]
        dx, dqw, dkw = qk_norm_bwd(x, heads, q_weight, k_weight, *grads, eps, rotary, positions, interleaved)
        return dx, dqw, dkw, None, None, None, None, None


def qk_norm(x, heads, q_weight=None, k_weight=None, eps: float = 1e-6, rotary=None, positions=None,
            interleaved: bool = False):
    """Differentiable norm of query and key heads with the position rotation:
    packed projection x [B, N, (Hq + Hk + Hv) * 64] -> (Q, K, V) as
    qk_norm_fwd (gradients reach x and the weights; captured as cross_attention)."""
    return QkNormFunction.apply(x, q_weight, k_weight, tuple(int(h) for h in heads), float(eps), rotary, positions,
                                bool(interleaved))


# --------------------------------------------------------- cross attention

_pack_heads = _native.HEADS.pack


def _heads_arg(name: str, t, shape, dtype, index: int) -> bytes:
    """t as a packed fibatt_heads."""
    try:
        good = t.dtype is dtype and t.get_device() == index and t.shape == shape
    except AttributeError:
        good = False
    if not good:
        _check_tensor(name, t, dtype, index)
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    sb, sh, sn, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must have contiguous rows")
    # a dim of one element has no stride that matters
    b, h, n, _ = shape
    return _pack_heads(t.data_ptr(), sb if b > 1 else 0, sh if h > 1 else 0, sn if n > 1 else 0)


def _numbers(name: str, t, B: int, index: int) -> int:
    """The address of one int32 a sequence."""
    try:
        if t.dtype is _INT32 and t.get_device() == index and t.shape == (B,) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _check_dense(name, t, (B,), _INT32, index)


_INT32 = torch.int32


def _attention_sizes(Q, K, V):
    """(dtype, its code, device index) of four-dim tensors Q, K, V."""
    try:
        dtype = Q.dtype
        if Q.dim() == 4 and K.dim() == 4 and V.dim() == 4 and Q.is_cuda:
            return dtype, _DTYPES[dtype], Q.get_device()
    except (AttributeError, KeyError):
        pass
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a [B, H, N, D] tensor")
    if Q.dtype not in _DTYPES:
        raise ValueError(f"dtype {Q.dtype} unsupported (float32 or bfloat16)")
    return Q.dtype, _DTYPES[Q.dtype], _index("Q", Q)


def _cross_desc(Q, K, V, scale, kv_len, key_mask):
    """(packed fibatt_cross, Q, K, V as packed fibatt_heads, device index)."""
    dtype, code, index = _attention_sizes(Q, K, V)
    B, Hq, Nq, D = shape = Q.shape
    _, Hkv, Nk, _ = K.shape
    lens = mask = mask_sb = 0
    if kv_len is not None:
        lens = _check_dense("kv_len", kv_len, (B,), torch.int32, index)
    if key_mask is not None:
        if not isinstance(key_mask, torch.Tensor) or key_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError("key_mask must be a bool or uint8 tensor")
        _check_tensor("key_mask", key_mask, key_mask.dtype, index)
        if key_mask.shape != (B, Nk) or (Nk > 1 and key_mask.stride(1) != 1):
            raise ValueError(f"key_mask must be [B, Nk] = {(B, Nk)} with contiguous rows, got {tuple(key_mask.shape)}")
        mask, mask_sb = key_mask.data_ptr(), key_mask.stride(0)
    kv_shape = (B, Hkv, Nk, D)
    return (_native.CROSS.pack(B, Hq, Hkv, Nq, Nk, D, code, scale, lens, mask, mask_sb),
            _heads_arg("Q", Q, shape, dtype, index), _heads_arg("K", K, kv_shape, dtype, index),
            _heads_arg("V", V, kv_shape, dtype, index), index)


def cross_fwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, scale: float, kv_len: torch.Tensor | None = None,
              key_mask: torch.Tensor | None = None, O: torch.Tensor | None = None, LSE: torch.Tensor | None = None,
              stream=None):
    """fibatt_cross_fwd: queries Q [B, Hq, Nq, 64] on keys and values K, V
    [B, Hkv, Nk, 64] (Hkv divides Hq; any strides whose rows are contiguous);
    returns (O, LSE), O in Q's layout.  kv_len: int32 [B], the keys each
    sequence has; key_mask: bool [B, Nk], the keys it attends."""
    d, q, k, v, index = _cross_desc(Q, K, V, scale, kv_len, key_mask)
    return _launch(index, stream, _attention_fwd, lib().fibatt_cross_fwd, d, q, k, v, Q, O, LSE, index)


def _attention_fwd(call, d, q, k, v, Q, O, LSE, index, s):
    shape = Q.shape
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None:
        LSE = torch.empty(shape[:3], dtype=torch.float32, device=Q.device)
        lse = LSE.data_ptr()
    else:
        lse = _check_dense("LSE", LSE, shape[:3], torch.float32, index)
    status = call(d, q, k, v, _heads_arg("O", O, shape, Q.dtype, index), lse, s)
    if status:
        check(status)
    return O, LSE


def cross_bwd(Q, K, V, O, LSE, dO, scale: float, kv_len=None, key_mask=None, dQ=None, dK=None, dV=None,
              workspace: torch.Tensor | None = None, stream=None):
    """fibatt_cross_bwd: (dQ, dK, dV) from cross_fwd's O and LSE and the
    gradient dO of O; each gradient in its input's layout unless given."""
    L = lib()
    return _attention_bwd(L.fibatt_cross_bwd, L.fibatt_cross_bwd_workspace_bytes,
                          _cross_desc(Q, K, V, scale, kv_len, key_mask), Q, K, V, O, LSE, dO, dQ, dK, dV, workspace, stream)


def _attention_bwd(bwd_call, workspace_bytes, desc, Q, K, V, O, LSE, dO, dQ, dK, dV, workspace, stream):
    d, q, k, v, index = desc
    shape, dtype = Q.shape, Q.dtype
    _check_dense("LSE", LSE, shape[:3], torch.float32, index)
    o, do = _heads_arg("O", O, shape, dtype, index), _heads_arg("dO", dO, shape, dtype, index)

    def call(s):
        dq = torch.empty_like(Q) if dQ is None else dQ
        dk = torch.empty_like(K) if dK is None else dK
        dv = torch.empty_like(V) if dV is None else dV
        ws = _workspace(workspace, workspace_bytes(d), index)
        check(bwd_call(d, q, k, v, o, LSE.data_ptr(), do, _heads_arg("dQ", dq, shape, dtype, index),
                       _heads_arg("dK", dk, K.shape, dtype, index), _heads_arg("dV", dv, K.shape, dtype, index),
                       ws.data_ptr(), ws.numel() * ws.element_size(), s))
        return dq, dk, dv

    return _launch(index, stream, call)


class CrossAttentionFunction(torch.autograd.Function):
    """Autograd wrapper: forward = fibatt_cross_fwd, backward = fibatt_cross_bwd."""

    @staticmethod
    def forward(ctx, Q, K, V, scale, kv_len, key_mask):
        Q, K, V = _readable(Q), _readable(K), _readable(V)
        O, LSE = cross_fwd(Q, K, V, scale, kv_len, key_mask)
        ctx.save_for_backward(Q, K, V, O, LSE, kv_len, key_mask)
        ctx.scale = scale
        return O

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        Q, K, V, O, LSE, kv_len, key_mask = ctx.saved_tensors
        dQ, dK, dV = cross_bwd(Q, K, V, O, LSE, _readable(dO), ctx.scale, kv_len, key_mask)
        return dQ, dK, dV, None, None, None


def cross_attention(Q, K, V, scale: float | None = None, kv_len=None, key_mask=None):
    """Differentiable cross attention: Q [B, Hq, Nq, 64] on K, V [B, Hkv, Nk, 64]
    (arguments as cross_fwd).  To capture a backward pass into a graph, capture
    its forward pass with it, with no eager graph of the same leaves alive: torch
    would make their gradients wait on the stream of the eager pass."""
    if scale is None:
        scale = Q.shape[-1] ** -0.5
    return CrossAttentionFunction.apply(Q, K, V, float(scale), kv_len, key_mask)


# ------------------------------------------ attention over a window, with sinks

# The calls below first try the short way in C++ (binding/calls.cpp), which takes those of the
# usual form; None from there: the steps here, which take every form and say what is wrong with a call.
_calls = None


def _short():
    global _calls
    _calls = _native.calls()
    return _calls


def _window_desc(Q, K, V, scale, window, sinks, q_start, kv_len):
    """(packed fibatt_window, Q, K, V as packed fibatt_heads, device index)."""
    dtype, code, index = _attention_sizes(Q, K, V)
    B, Hq, Nq, D = shape = Q.shape
    _, Hkv, Nk, _ = K.shape
    window, sinks = _band(window, sinks)
    kv_shape = (B, Hkv, Nk, D)
    return (_native.WINDOW.pack(B, Hq, Hkv, Nq, Nk, D, code, scale, window, sinks,
                                0 if q_start is None else _numbers("q_start", q_start, B, index),
                                0 if kv_len is None else _numbers("kv_len", kv_len, B, index)),
            _heads_arg("Q", Q, shape, dtype, index), _heads_arg("K", K, kv_shape, dtype, index),
            _heads_arg("V", V, kv_shape, dtype, index), index)


def _band(window, sinks):
    """(window, sinks) as the library takes them: no window is one that holds every key."""
    return _ALL if window is None else min(operator.index(window), _ALL), min(operator.index(sinks), _ALL)


_ALL = 2**31 - 1


def window_fwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, scale: float, window: int | None = None, sinks: int = 0,
               q_start: torch.Tensor | None = None, kv_len: torch.Tensor | None = None, O: torch.Tensor | None = None,
               LSE: torch.Tensor | None = None, stream=None):
    """fibatt_window_fwd: causal attention of Q [B, Hq, Nq, 64] to K, V [B, Hkv,
    Nk, 64] (Hkv divides Hq; any strides whose rows are contiguous), each query
    to the `window` keys up to its own place (None: all) and to the first `sinks`; returns (O, LSE),
    O in Q's layout.  q_start: int32 [B], the place of each sequence's first
    query (Nk - Nq if not given); kv_len: int32 [B], the keys each sequence
    has.  Queries outside their sequence attend nothing: O = 0, LSE = -inf."""
    if O is None and LSE is None and stream is None:
        r = (_calls or _short()).window_fwd(Q, K, V, scale, window, sinks, q_start, kv_len)
        if r.__class__ is tuple:
            return r
        if r is not None:
            check(r)
    d, q, k, v, index = _window_desc(Q, K, V, scale, window, sinks, q_start, kv_len)
    return _launch(index, stream, _attention_fwd, lib().fibatt_window_fwd, d, q, k, v, Q, O, LSE, index)


def window_bwd(Q, K, V, O, LSE, dO, scale: float, window: int | None = None, sinks: int = 0, q_start=None, kv_len=None,
               dQ=None, dK=None, dV=None, workspace: torch.Tensor | None = None, stream=None):
    """fibatt_window_bwd: (dQ, dK, dV) from window_fwd's O and LSE and the
    gradient dO of O; each gradient in its input's layout unless given."""
    if dQ is None and dK is None and dV is None and workspace is None and stream is None:
        r = (_calls or _short()).window_bwd(Q, K, V, O, LSE, dO, scale, window, sinks, q_start, kv_len)
        if r.__class__ is tuple:
            return r
        if r is not None:
            check(r)
    L = lib()
    return _attention_bwd(L.fibatt_window_bwd, L.fibatt_window_bwd_workspace_bytes,
                          _window_desc(Q, K, V, scale, window, sinks, q_start, kv_len), Q, K, V, O, LSE, dO, dQ, dK, dV,
                          workspace, stream)


class WindowAttentionFunction(torch.autograd.Function):
    """Autograd wrapper: forward = fibatt_window_fwd, backward = fibatt_window_bwd."""

    @staticmethod
    def forward(ctx, Q, K, V, scale, window, sinks, q_start, kv_len):
        Q, K, V = _readable(Q), _readable(K), _readable(V)
        O, LSE = window_fwd(Q, K, V, scale, window, sinks, q_start, kv_len)
        ctx.save_for_backward(Q, K, V, O, LSE, q_start, kv_len)
        ctx.how = (scale, window, sinks)
        return O

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        Q, K, V, O, LSE, q_start, kv_len = ctx.saved_tensors
        dQ, dK, dV = window_bwd(Q, K, V, O, LSE, _readable(dO), *ctx.how, q_start, kv_len)
        return dQ, dK, dV, None, None, None, None, None


def window_attention(Q, K, V, scale: float | None = None, window: int | None = None, sinks: int = 0, q_start=None,
                     kv_len=None):
    """Differentiable attention over a window with sinks (arguments as window_fwd; captured
    as cross_attention)."""
    if scale is None:
        scale = Q.shape[-1] ** -0.5
    return WindowAttentionFunction.apply(Q, K, V, float(scale), window, sinks, q_start, kv_len)


# ------------------------------------------------ paged cache in 8 bits

PAGE = 64                    # tokens of a page


class Cache(NamedTuple):
    """A cache's memory: data [pages, Hkv, 2, 4096] uint8 (a page's keys
    [64 tokens][64 dims], then its values [64 dims][64 tokens], as e4m3) and
    scales [pages, Hkv, 2] fp32.  Which sequence has which pages is a table that
    the caller keeps: int32 [B, pages of a sequence]."""

    data: torch.Tensor
    scales: torch.Tensor

    @classmethod
    def new(cls, pages: int, kv_heads: int, device=None) -> "Cache":
        """A cache of so many pages, of 64 tokens each."""
        device = torch.device("cuda") if device is None else device
        return cls(torch.zeros(pages, kv_heads, 2, PAGE * HEAD_DIM, dtype=torch.uint8, device=device),
                   torch.ones(pages, kv_heads, 2, device=device))


def _cache_desc(cache, table, start, count, dtype, B, N, D, index):
    """(packed fibatt_cache, key heads)."""
    data, scales = cache
    try:
        code = _DTYPES[dtype]
        pages, Hkv, two, piece = data.shape
        rows, entries = table.shape
        good = (data.dtype is torch.uint8 and data.get_device() == index and (two, piece) == _CACHE_SHAPE
                and data.is_contiguous() and scales.dtype is torch.float32 and scales.get_device() == index
                and scales.shape == (pages, Hkv, 2) and scales.is_contiguous()
                and table.dtype is _INT32 and table.get_device() == index and rows == B
                and (entries == 1 or table.stride(1) == 1))
    except (AttributeError, KeyError, ValueError):
        good = False
    if not good:
        _refuse_cache(data, scales, table, dtype, B, index)
    return _native.CACHE.pack(B, Hkv, N, D, code, pages, entries, data.data_ptr(), scales.data_ptr(), table.data_ptr(),
                              table.stride(0) if B > 1 else 0,
                              0 if start is None else _numbers("start", start, B, index),
                              0 if count is None else _numbers("count", count, B, index)), Hkv


def _refuse_cache(data, scales, table, dtype, B, index):
    if dtype not in _DTYPES:
        raise ValueError(f"dtype {dtype} unsupported (float32 or bfloat16)")
    _check_tensor("data", data, torch.uint8, index)
    if data.dim() != 4 or data.shape[2:] != _CACHE_SHAPE or not data.is_contiguous():
        raise ValueError(f"data must be a contiguous [pages, Hkv, 2, {PAGE * HEAD_DIM}] tensor, got {tuple(data.shape)}")
    _check_dense("scales", scales, (*data.shape[:2], 2), torch.float32, index)
    _check_tensor("table", table, _INT32, index)
    raise ValueError(f"table must be [B, pages of a sequence] with B={B} and contiguous rows, got {tuple(table.shape)}")


_CACHE_SHAPE = (2, PAGE * HEAD_DIM)


def _cache_states(cache, table, K, V, start, count):
    """(packed fibatt_cache, K, V as packed fibatt_heads, device index)."""
    for name, t in (("K", K), ("V", V)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a [B, H, N, D] tensor")
    index = _index("K", K)
    B, _, N, D = K.shape
    d, Hkv = _cache_desc(cache, table, start, count, K.dtype, B, N, D, index)
    shape = (B, Hkv, N, D)
    return d, _heads_arg("K", K, shape, K.dtype, index), _heads_arg("V", V, shape, K.dtype, index), index


def cache_store(cache: Cache, table: torch.Tensor, K: torch.Tensor, V: torch.Tensor, start: torch.Tensor | None = None,
                count: torch.Tensor | None = None, stream=None) -> None:
    """fibatt_cache_store: keys and values K, V [B, Hkv, N, 64] of N tokens into
    the sequences' pages, token n of them at place start[b] + n (int32 [B]; from 0
    if not given); count: int32 [B], how many of the N each sequence has."""
    if stream is None:
        r = (_calls or _short()).cache_store(*cache, table, K, V, start, count)
        if r is not None:
            return check(r)
    d, k, v, index = _cache_states(cache, table, K, V, start, count)
    check(_launch(index, stream, lib().fibatt_cache_store, d, k, v))


def cache_load(cache: Cache, table: torch.Tensor, N: int, start: torch.Tensor | None = None,
               count: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16, K: torch.Tensor | None = None,
               V: torch.Tensor | None = None, stream=None):
    """fibatt_cache_load: (K, V), [B, Hkv, N, 64] each, of the N tokens from
    place start[b] on, zeros from count[b] on."""
    if K is None and V is None and stream is None and dtype in _DTYPES:
        r = (_calls or _short()).cache_load(*cache, table, N, start, count, dtype is torch.float32)
        if r.__class__ is tuple:
            return r
        if r is not None:
            check(r)
    index = _index("data", cache[0])
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [B, pages of a sequence]")
    shape = (table.shape[0], cache[0].shape[1], operator.index(N), HEAD_DIM)
    if K is not None:
        dtype = K.dtype
    d, _ = _cache_desc(cache, table, start, count, dtype, shape[0], shape[2], HEAD_DIM, index)

    def call(s):
        k = torch.empty(shape, dtype=dtype, device=cache[0].device) if K is None else K
        v = torch.empty(shape, dtype=dtype, device=cache[0].device) if V is None else V
        check(lib().fibatt_cache_load(d, _heads_arg("K", k, shape, dtype, index), _heads_arg("V", v, shape, dtype, index), s))
        return k, v

    return _launch(index, stream, call)


def cache_fwd(Q: torch.Tensor, cache: Cache, table: torch.Tensor, start: torch.Tensor | None, scale: float,
              window: int | None = None, sinks: int = 0, count: torch.Tensor | None = None, O: torch.Tensor | None = None,
              LSE: torch.Tensor | None = None, stream=None):
    """fibatt_cache_fwd: attention of Q [B, Hq, N, 64], the queries of the tokens
    at start[b] + n, to the cache that holds their keys (cache_store comes
    first); window, sinks as window_fwd; returns (O, LSE), O in Q's layout.  A
    query that count[b] leaves out attends nothing: O = 0, LSE = -inf."""
    if O is None and LSE is None and stream is None:
        r = (_calls or _short()).cache_fwd(Q, *cache, table, start, scale, window, sinks, count)
        if r.__class__ is tuple:
            return r
        if r is not None:
            check(r)
    dtype, _, index = _attention_sizes(Q, Q, Q)
    B, Hq, N, D = shape = Q.shape
    d, _ = _cache_desc(cache, table, start, count, dtype, B, N, D, index)
    return _launch(index, stream, _cache_fwd, d, Hq, scale, *_band(window, sinks), _heads_arg("Q", Q, shape, dtype, index),
                   Q, O, LSE, index)


def _cache_fwd(d, Hq, scale, window, sinks, q, Q, O, LSE, index, s):
    shape = Q.shape
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None:
        LSE = torch.empty(shape[:3], dtype=torch.float32, device=Q.device)
        lse = LSE.data_ptr()
    else:
        lse = _check_dense("LSE", LSE, shape[:3], torch.float32, index)
    status = lib().fibatt_cache_fwd(d, Hq, scale, window, sinks, q, _heads_arg("O", O, shape, Q.dtype, index), lse, s)
    if status:
        check(status)
    return O, LSE


__all__ = ["FibattError", "Support", "fwd", "bwd", "bwd_noalloc", "fibottention", "FibottentionFunction",
           "qk_norm_fwd", "qk_norm_bwd", "qk_norm", "QkNormFunction", "rotary_tables", "rotary_angles",
           "rotary_angles_2d", "cross_fwd", "cross_bwd", "cross_attention", "CrossAttentionFunction",
           "window_fwd", "window_bwd", "window_attention", "WindowAttentionFunction",
           "Cache", "cache_store", "cache_load", "cache_fwd", "PAGE",
           "wythoff_row", "wythoff_row_modified", "window_schedule", "HEAD_DIM"]
