"""A drop-in multi-head self-attention layer whose attention core is
Fibottention (the paper's Sec. 3 applied in a ViT encoder block: the QKV
projection, per-head attention over the Fibonacci support, the output
projection W^Z; README Algorithm 3 shows the same sequence of steps).

The projections are ordinary torch GEMMs; the attention core calls libfibatt
through ``fibottention`` (forward fibatt_fwd, backward fibatt_bwd).  Head i of
the layer uses Wythoff row pi(i) with the linear window schedule (paper
Sec. 3: a per-layer permutation pi of the heads is allowed).  Query/key norms
and a position rotation can go between the projection and the attention, and
``CrossAttention`` is a decoder's layer on such an encoder's states.
"""
from __future__ import annotations

import torch
from torch import nn

from .api import HEAD_DIM, Support, cross_attention, fibottention, qk_norm, rotary_tables


class _Rotary(nn.Module):
    """cos and sin tables, which keep their 32 bits when the layer's type
    changes (the angles of far positions do not survive 16)."""

    def __init__(self, angles: torch.Tensor):
        super().__init__()
        self.cos, self.sin = rotary_tables(angles)

    def _apply(self, fn, recurse=True):
        dev = fn(torch.empty(0, device=self.cos.device)).device
        self.cos, self.sin = self.cos.to(dev), self.sin.to(dev)
        return self

    def tables(self):
        return self.cos, self.sin


def _weight(w, x: torch.Tensor):
    """A norm's weight (or None) in the type of the projection x: under autocast x
    has 16 bits and the parameter 32, and it is rounded as the projection's own
    weights are (its gradient comes back through the cast)."""
    return None if w is None else w.to(x.dtype)


def _turned(rotary, positions):
    """(tables, positions) for qk_norm; neither for a layer that does not rotate."""
    return (None, None) if rotary is None else (rotary.tables(), positions)


class FibottentionSelfAttention(nn.Module):
    """x [B, N, dim] -> [B, N, dim] with dim = heads * 64.

    norm: RMS norm of every query and key head (weights q_norm, k_norm; eps).
    rotary: position rotation by the angles of a table [positions, pairs]
    (api.rotary_angles, rotary_angles_2d); with class_token, token 0 is not
    rotated and token n is at position n - 1.  Either runs with the split into
    heads in one pass (api.qk_norm)."""

    def __init__(self, dim: int, heads: int, N: int, w_min: int, w_max: int, include_diag: bool = True,
                 global_token: bool = False, modified: bool = False, permutation=None, bias: bool = True,
                 norm: bool = False, rotary: torch.Tensor | None = None, class_token: bool = False, eps: float = 1e-6):
        super().__init__()
        if dim != heads * HEAD_DIM:
            raise ValueError(f"dim must be heads * {HEAD_DIM}")
        self.heads, self.N = heads, N
        self.qkv = nn.Linear(dim, 3 * dim, bias=bias)
        self.proj = nn.Linear(dim, dim, bias=bias)
        self.support = Support.wythoff(heads, N, w_min, w_max, include_diag, modified=modified,
                                       permutation=permutation).set_global_token(global_token)
        self.scale = HEAD_DIM ** -0.5
        self.q_norm = nn.Parameter(torch.ones(HEAD_DIM)) if norm else None
        self.k_norm = nn.Parameter(torch.ones(HEAD_DIM)) if norm else None
        self.eps = eps
        self.rotary = None if rotary is None else _Rotary(rotary)
        first = 1 if class_token else 0
        if rotary is not None and rotary.shape[0] < N - first:
            raise ValueError(f"rotary has {rotary.shape[0]} positions, the layer {N - first}")
        self.register_buffer("positions", torch.arange(N, dtype=torch.int32) - first if class_token and rotary is not None
                             else None, persistent=False)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        B, N, dim = x.shape
        if N != self.N:
            raise ValueError(f"sequence length {N}, layer built for {self.N}")
        qkv = self.qkv(x)
        if self.q_norm is not None or self.rotary is not None:
            q, k, v = qk_norm(qkv, (self.heads,) * 3, _weight(self.q_norm, qkv), _weight(self.k_norm, qkv), self.eps,
                              None if self.rotary is None else self.rotary.tables(), self.positions)
        else:
            qkv = qkv.view(B, N, 3, self.heads, HEAD_DIM).permute(2, 0, 3, 1, 4)
            q, k, v = (t.contiguous() for t in qkv)            # [B, H, N, 64] each
        o = fibottention(q, k, v, self.support, self.scale)  # [B, H, N, 64]
        return self.proj(o.transpose(1, 2).reshape(B, N, dim))


class CrossAttention(nn.Module):
    """Decoder tokens x [B, Nq, dim] on an encoder's states y [B, Nk, state_dim]
    -> [B, Nq, dim], dim = heads * 64: the decoder's layer beside an encoder of
    FibottentionSelfAttention layers.

    kv_heads: key/value heads, shared by heads / kv_heads query heads each.
    norm: RMS norm of every query and key head.  rotary, state_rotary: tables
    of angles for the decoder's and the encoder's positions (None: not
    rotated).  states() computes an encoder's keys and values once, for
    decoding many tokens against them."""

    def __init__(self, dim: int, heads: int, state_dim: int | None = None, kv_heads: int | None = None,
                 bias: bool = True, norm: bool = False, rotary: torch.Tensor | None = None,
                 state_rotary: torch.Tensor | None = None, eps: float = 1e-6):
        super().__init__()
        if dim != heads * HEAD_DIM:
            raise ValueError(f"dim must be heads * {HEAD_DIM}")
        self.heads = heads
        self.kv_heads = heads if kv_heads is None else kv_heads
        if self.kv_heads < 1 or heads % self.kv_heads:
            raise ValueError(f"kv_heads {kv_heads} does not divide {heads} heads")
        self.q = nn.Linear(dim, dim, bias=bias)
        self.kv = nn.Linear(dim if state_dim is None else state_dim, 2 * self.kv_heads * HEAD_DIM, bias=bias)
        self.proj = nn.Linear(dim, dim, bias=bias)
        self.scale = HEAD_DIM ** -0.5
        self.q_norm = nn.Parameter(torch.ones(HEAD_DIM)) if norm else None
        self.k_norm = nn.Parameter(torch.ones(HEAD_DIM)) if norm else None
        self.eps = eps
        self.rotary = None if rotary is None else _Rotary(rotary)
        self.state_rotary = None if state_rotary is None else _Rotary(state_rotary)

    def states(self, y: torch.Tensor, positions: torch.Tensor | None = None):
        """Keys and values [B, kv_heads, Nk, 64] of the encoder's states; positions
        (int32 [Nk] or [B, Nk]): their places, 0.. if not given, -1 for a class token."""
        kv = self.kv(y)
        return qk_norm(kv, (0, self.kv_heads, self.kv_heads), None, _weight(self.k_norm, kv), self.eps,
                       *_turned(self.state_rotary, positions))[1:]

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, kv_len: torch.Tensor | None = None,
                key_mask: torch.Tensor | None = None, positions: torch.Tensor | None = None, kv=None) -> torch.Tensor:
        """y: the states, at positions 0.., or kv: what states() made of them (which
        takes positions of their own); kv_len [B] int32 and key_mask [B, Nk] say
        which of them each sequence attends; positions (int32 [Nq] or [B, Nq]): the
        decoder tokens' places, 0.. if not given (without rotary they make no
        difference)."""
        if (y is None) == (kv is None):
            raise ValueError("either the states y or their kv")
        B, Nq, dim = x.shape
        k, v = self.states(y) if kv is None else kv
        q = self.q(x)
        if self.q_norm is not None or self.rotary is not None:
            q = qk_norm(q, (self.heads, 0, 0), _weight(self.q_norm, q), None, self.eps, *_turned(self.rotary, positions))[0]
        else:
            q = q.view(B, Nq, self.heads, HEAD_DIM).transpose(1, 2)
        o = cross_attention(q, k, v, self.scale, kv_len, key_mask)     # [B, H, Nq, 64], in q's layout
        return self.proj(o.transpose(1, 2).reshape(B, Nq, dim))


__all__ = ["FibottentionSelfAttention", "CrossAttention"]
