"""A drop-in multi-head self-attention layer whose attention core is
Fibottention (the paper's Sec. 3 applied in a ViT encoder block: the QKV
projection, per-head attention over the Fibonacci support, the output
projection W^Z; README Algorithm 3 shows the same sequence of steps).

The projections are ordinary torch GEMMs; the attention core calls libfibatt
through ``fibottention`` (forward fibatt_fwd, backward fibatt_bwd).  Head i of
the layer uses Wythoff row pi(i) with the linear window schedule (paper
Sec. 3: a per-layer permutation pi of the heads is allowed).  Query/key norms
and a position rotation can go between the projection and the attention, and
``CrossAttention`` is a decoder's layer on such an encoder's states,
``WindowSelfAttention`` one on the decoder's own tokens.
"""
from __future__ import annotations

import torch
from torch import nn

from .api import (HEAD_DIM, PAGE, Support, cache_fwd, cache_load, cache_store, cross_attention, fibottention, qk_norm,
                  rotary_tables, window_attention, window_fwd)


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


class WindowSelfAttention(nn.Module):
    """Decoder tokens x [B, N, dim] on themselves -> [B, N, dim], dim = heads *
    64: causal, each token on the `window` tokens up to itself (None: all) and on the
    first `sinks`.

    kv_heads: key/value heads, shared by heads / kv_heads query heads each.
    norm: RMS norm of every query and key head.  rotary: a table of angles for the
    tokens' places (None: not rotated).  forward() is for whole sequences, in
    training; step() decodes on a paged 8-bit cache (api.Cache)."""

    def __init__(self, dim: int, heads: int, kv_heads: int | None = None, window: int | None = None, sinks: int = 0,
                 bias: bool = True, norm: bool = False, rotary: torch.Tensor | None = None, eps: float = 1e-6):
        super().__init__()
        if dim != heads * HEAD_DIM:
            raise ValueError(f"dim must be heads * {HEAD_DIM}")
        self.heads = heads
        self.kv_heads = heads if kv_heads is None else kv_heads
        if self.kv_heads < 1 or heads % self.kv_heads:
            raise ValueError(f"kv_heads {kv_heads} does not divide {heads} heads")
        if (window is not None and window < 1) or sinks < 0:
            raise ValueError(f"window {window} must be at least 1, sinks {sinks} at least 0")
        self.window, self.sinks = window, sinks
        self.qkv = nn.Linear(dim, (heads + 2 * self.kv_heads) * HEAD_DIM, bias=bias)
        self.proj = nn.Linear(dim, dim, bias=bias)
        self.scale = HEAD_DIM ** -0.5
        self.q_norm = nn.Parameter(torch.ones(HEAD_DIM)) if norm else None
        self.k_norm = nn.Parameter(torch.ones(HEAD_DIM)) if norm else None
        self.eps = eps
        self.rotary = None if rotary is None else _Rotary(rotary)

    def _split(self, x, positions):
        """Queries, keys and values [B, H, N, 64] of the tokens x."""
        heads = (self.heads, self.kv_heads, self.kv_heads)
        qkv = self.qkv(x)
        if self.q_norm is None and self.rotary is None:
            qkv = qkv.unflatten(-1, (sum(heads), HEAD_DIM)).transpose(1, 2)
            return qkv.split(heads, 1)
        return qk_norm(qkv, heads, _weight(self.q_norm, qkv), _weight(self.k_norm, qkv), self.eps,
                       *_turned(self.rotary, positions))

    def _join(self, o):
        return self.proj(o.transpose(1, 2).flatten(2))

    def forward(self, x: torch.Tensor, kv_len: torch.Tensor | None = None) -> torch.Tensor:
        """kv_len [B] int32: the sequences' lengths where they are padded behind (the
        padding's outputs are the projection's bias)."""
        q, k, v = self._split(x, None)
        return self._join(window_attention(q, k, v, self.scale, self.window, self.sinks, None, kv_len))

    @torch.no_grad()
    def step(self, x: torch.Tensor, cache, table: torch.Tensor, start: torch.Tensor,
             count: torch.Tensor | None = None) -> torch.Tensor:
        """The next N tokens x [B, N, dim] of sequences that have start[b] tokens in
        `cache` (int32 [B]; the table [B, pages] has pages for the new ones too), into
        which theirs go.  count [B] int32: how many of the N each sequence has.
        Without gradients; start is the caller's to move on.  Pages of tokens that the window has left behind, and
        that are no sinks', may be given back.  Many tokens at once on a layer without a window take
        scratch memory for the keys and values of as many tokens as the table has places for; with one, for
        those of the window, the sinks and the new tokens."""
        N = x.shape[1]
        places = start[:, None] + torch.arange(N, dtype=torch.int32, device=x.device)
        held = start + (N if count is None else count.clamp(0, N))
        if count is not None:      # tokens that are left out stand at the last place that there is
            places = torch.minimum(places, held[:, None] - 1)
        q, k, v = self._split(x, places)
        cache_store(cache, table, k, v, start, count)
        if self._page_by_page(x.shape[0], N, table.shape[1] * PAGE, q.dtype):
            return self._join(cache_fwd(q, cache, table, start, self.scale, self.window, self.sinks, count)[0])
        return self._join(self._attend_loaded(q, cache, table, start, held))

    def _page_by_page(self, B, N, places, dtype):
        """Whether the queries of N tokens attend the cache's pages as they are, 16 rows of a key head at a
        time (_attend_loaded's way otherwise).

        In 32 bits always: the products of the loaded tokens cost more than the pages read again (8 sequences,
        16 heads on 4, 1024 rows, 16448 places: window 1024 126 us and 245, none 799 and 2858; at worst, 32
        sequences, window 128: 259 and 201).  In 16 bits where an estimate says so, in ns: a block of 16
        rows costs 15, and 1.1 a page that it reads; loading 20000, and 0.16 a token and head; without a
        window all of the table's places are taken to be held.  (us, pages and loaded, 16
        heads on 4; 1 sequence, 16448 places, no window, 512 rows 28.7 and 34.2, 1024 rows 49.5 and 35.3;
        8 sequences, window 128, 256 rows 13.0 and 21.2, 512 rows 22.4 and 22.1; window 1024 22.5 and 30.7, 38.9
        and 31.9; no window, 128 rows 75.5 and 89.5, 256 rows 139 and 119; 32 sequences, window 1024, 128 rows 38.7
        and 39.6, 256 rows 73.5 and 44.8.)"""
        if dtype == torch.float32:
            return True
        heads, rows = B * self.kv_heads, self.heads // self.kv_heads * N
        seen = places if self.window is None else min(places, self.window + self.sinks)
        loaded = places if self.window is None else min(places, self.window + self.sinks + N)
        return heads * ((rows + 15) // 16) * (15 + 1.1 * seen / PAGE) <= 20000 + 0.16 * heads * loaded

    def _attend_loaded(self, q, cache, table, start, held):
        """Attention of the queries from place start[b] on to the cache's tokens, up to held[b], as 16
        or 32 bits.  With a window the tokens that are attended alone: those of the sinks, and behind
        them those from the oldest key that the first query's window reaches on, so that the queries' places in
        what is loaded are their own less what lies between.  Entries of the table that no query needs
        are not looked at, and what is loaded does not grow with the table."""
        B, _, N, _ = q.shape
        places = table.shape[1] * PAGE
        held = torch.where(held > start, held.clamp(max=places), 0)       # (a sequence without tokens needs no pages)
        if self.window is None or self.sinks >= places:
            k, v = cache_load(cache, table, places, None, held, dtype=q.dtype)
            return window_fwd(q, k, v, self.scale, self.window, self.sinks, start, held)[0]
        S, last = self.sinks, min(self.window + N - 1, places - self.sinks)
        oldest = (start.clamp(min=-N) - (self.window - 1)).clamp(min=S)
        k, v = (q.new_empty(B, self.kv_heads, S + last, HEAD_DIM) for _ in range(2))
        if S:
            cache_load(cache, table, S, None, held, K=k[:, :, :S], V=v[:, :, :S])
        n = held - oldest
        cache_load(cache, table, last, oldest, n, K=k[:, :, S:], V=v[:, :, S:])
        return window_fwd(q, k, v, self.scale, self.window, S, start - oldest + S, n + S)[0]


__all__ = ["FibottentionSelfAttention", "CrossAttention", "WindowSelfAttention"]
