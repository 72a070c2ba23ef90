"""Attention over a paged cache that holds keys and values in 4 bits (the
bitlinear_kv4_* calls of include/bitlinear.h): the part of a decoder block between
its Q/K/V projections and its output projection.

A batch is three int32 device tensors: ``q_start`` [S + 1] (rows of each
sequence's new tokens), ``kv_len`` [S] (tokens in the cache, the new ones
included) and ``page_table`` [S, W]. One token a sequence (decoding), a few, or
whole prompts go through the same calls, also mixed::

    cache = kv4_cache(num_pages, kv_heads, page_size, head_dim, device)
    q = kv4_append(q, k, v, cos_sin, cache, page_table, kv_len, q_start)
    o = kv4_attention(q, cache, page_table, kv_len, q_start, max_q)

Argument marshalling only, like the rest of the binding (compiled: csrc/native.cpp).
Calls run on the current stream of the tensors' device; scratch is allocated per
call, so calls on different streams, and captured graphs, never share any.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as _b

GROUP = 32  # dims that share a quantisation step


class Kv4Cache:
    """The four arrays of a cache: codes uint8 [num_pages, kv_heads, page_size, head_dim / 2] and
    steps bf16 [num_pages, kv_heads, page_size, head_dim / 32], of the keys and of the values."""

    __slots__ = ("k_codes", "k_steps", "v_codes", "v_steps", "kv_heads", "head_dim")

    def __init__(self, k_codes: torch.Tensor, k_steps: torch.Tensor, v_codes: torch.Tensor, v_steps: torch.Tensor):
        self.kv_heads, self.head_dim = _b.native().kv4_check(k_codes, k_steps, v_codes, v_steps)
        self.k_codes, self.k_steps, self.v_codes, self.v_steps = k_codes, k_steps, v_codes, v_steps


def kv4_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int, device) -> Kv4Cache:
    """An empty cache (zeroed)."""
    codes = (num_pages, kv_heads, page_size, head_dim // 2)
    steps = (num_pages, kv_heads, page_size, head_dim // GROUP)
    return Kv4Cache(torch.zeros(codes, dtype=torch.uint8, device=device),
                    torch.zeros(steps, dtype=torch.bfloat16, device=device),
                    torch.zeros(codes, dtype=torch.uint8, device=device),
                    torch.zeros(steps, dtype=torch.bfloat16, device=device))


def kv4_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos_sin: torch.Tensor, cache: Kv4Cache,
               page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor, interleaved: bool = False,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate q and k [M, heads, D] bf16 by their positions' rows of cos_sin [max_pos, D] fp32 (D/2 cosines, D/2 sines),
    store k and v in the cache and return the rotated q (in `out`, which may be q). Rows without a sequence or a position are
    left as they are in `out`."""
    r = _b.native().kv4_append(q, k, v, cos_sin, cache.k_codes, cache.k_steps, cache.v_codes, cache.v_steps, page_table,
                               kv_len, q_start, interleaved, out)
    if type(r) is int:
        _b._check(r, "bitlinear_kv4_append")
    return r


def kv4_read(cache: Kv4Cache, page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor, rows: int):
    """The cached values of the batch's tokens: (k, v), bf16 [rows, kv_heads, D]; rows without a token are not set."""
    r = _b.native().kv4_read(cache.k_codes, cache.k_steps, cache.v_codes, cache.v_steps, page_table, kv_len, q_start, rows)
    if type(r) is int:
        _b._check(r, "bitlinear_kv4_read")
    return r


def kv4_attention(q: torch.Tensor, cache: Kv4Cache, page_table: torch.Tensor, kv_len: torch.Tensor,
                  q_start: torch.Tensor, max_q: int, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of the batch's tokens q [M, Hq, D] bf16 over the cache (their own keys stored before):
    bf16 [M, Hq, D]. max_q: the largest number of new tokens of a sequence; it chooses the kernel for the whole batch, so a
    prompt beside single tokens slows these down. scale: 1 / sqrt(D) by default, 2^-100 to 2^100. Rows without a sequence are
    left as they are in `out`, which must not overlap q."""
    r = _b.native().kv4_attention(q, cache.k_codes, cache.k_steps, cache.v_codes, cache.v_steps, page_table, kv_len,
                                  q_start, max_q, scale, out, ws)
    if type(r) is int:
        _b._check(r, "bitlinear_kv4_attention")
    return r
