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

Argument marshalling only, like the rest of the binding. Calls run on the current
stream of the tensors' device; scratch is allocated per call, so calls on
different streams, and captured graphs, never share any.
"""
from __future__ import annotations

import functools
import struct
from contextlib import nullcontext
from typing import Optional

import torch

from . import binding as _b

GROUP = 32  # dims that share a quantisation step

# bl_kv4_cache and bl_kv4_batch of include/bitlinear.h, as the bytes that the C calls take a pointer to
_pack_cache = struct.Struct("=QQQQqiiii").pack  # four pointers, pages, page size, heads, head dim, padding
_pack_batch = struct.Struct("=QQQqii").pack     # three pointers, table stride, S, W

_BF16 = torch.bfloat16
_workspace_bytes = functools.lru_cache(maxsize=4096)(_b.workspace_bytes)


class Kv4Cache:
    """The four arrays of a cache: codes uint8 [num_pages, kv_heads, page_size, head_dim / 2] and
    steps bf16 [num_pages, kv_heads, page_size, head_dim / 32], of the keys and of the values."""

    __slots__ = ("k_codes", "k_steps", "v_codes", "v_steps", "kv_heads", "head_dim", "_c", "_index")

    def __init__(self, k_codes: torch.Tensor, k_steps: torch.Tensor, v_codes: torch.Tensor, v_steps: torch.Tensor):
        if not k_codes.is_cuda:
            raise ValueError("k_codes must be a CUDA tensor")
        if k_codes.dim() != 4:
            raise ValueError("codes must be [num_pages, kv_heads, page_size, head_dim / 2]")
        codes = k_codes.shape
        pages, heads, size, half = codes
        steps = (pages, heads, size, 2 * half // GROUP)
        index = k_codes.get_device()
        for t, name, dtype, shape in ((k_codes, "k_codes", torch.uint8, codes), (v_codes, "v_codes", torch.uint8, codes),
                                      (k_steps, "k_steps", _BF16, steps), (v_steps, "v_steps", _BF16, steps)):
            if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on cuda:{index}")
        self.k_codes, self.k_steps, self.v_codes, self.v_steps = k_codes, k_steps, v_codes, v_steps
        self.kv_heads, self.head_dim, self._index = heads, 2 * half, index
        self._c = _pack_cache(k_codes.data_ptr(), k_steps.data_ptr(), v_codes.data_ptr(), v_steps.data_ptr(), pages, size,
                              heads, 2 * half, 0)


def kv4_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int, device) -> Kv4Cache:
    """An empty cache (zeroed)."""
    codes = (num_pages, kv_heads, page_size, head_dim // 2)
    steps = (num_pages, kv_heads, page_size, head_dim // GROUP)
    return Kv4Cache(torch.zeros(codes, dtype=torch.uint8, device=device),
                    torch.zeros(steps, dtype=_BF16, device=device),
                    torch.zeros(codes, dtype=torch.uint8, device=device),
                    torch.zeros(steps, dtype=_BF16, device=device))


def _on(index: int):
    """The device of a call made current for it."""
    return _HERE if index == torch.cuda.current_device() else torch.cuda.device(index)


_HERE = nullcontext()


def _batch(index: int, page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor) -> bytes:
    for t, name in ((kv_len, "kv_len"), (q_start, "q_start"), (page_table, "page_table")):
        if t.dtype is not torch.int32 or t.get_device() != index:
            raise ValueError(f"{name} must be an int32 tensor on cuda:{index}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [S, W]")
    S, W = page_table.shape
    stride, unit = page_table.stride()
    if unit != 1 and W > 1:
        raise ValueError("page_table must have contiguous rows")
    if kv_len.shape != (S,) or q_start.shape != (S + 1,) or not kv_len.is_contiguous() or not q_start.is_contiguous():
        raise ValueError(f"kv_len must be [{S}] and q_start [{S + 1}], contiguous")
    return _pack_batch(q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), stride, S, W)


def _rows(t: torch.Tensor, name: str, M: int, heads: int, D: int, index: int) -> int:
    """Row stride of t [M, heads, D] bf16 with the heads of a row side by side."""
    if t.dtype is not _BF16 or t.get_device() != index or t.shape != (M, heads, D):
        raise ValueError(f"{name} must be a bf16 tensor ({M}, {heads}, {D}) on cuda:{index}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    row, head, unit = t.stride()
    if unit != 1 or (head != D and heads > 1):
        raise ValueError(f"{name} must have the heads of a row side by side")
    return row if M > 1 else heads * D  # the stride of a single row means nothing


def kv4_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos_sin: torch.Tensor, cache: Kv4Cache,
               page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor, interleaved: bool = False,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate q and k [M, heads, D] bf16 by their positions' rows of cos_sin [max_pos, D] fp32 (D/2 cosines, D/2 sines),
    store k and v in the cache and return the rotated q (in `out`, which may be q)."""
    D, hkv, index = cache.head_dim, cache.kv_heads, cache._index
    M, Hq, _ = q.shape
    batch = _batch(index, page_table, kv_len, q_start)
    qs = _rows(q, "q", M, Hq, D, index)
    ks = _rows(k, "k", M, hkv, D, index)
    vs = _rows(v, "v", M, hkv, D, index)
    if (cos_sin.dtype is not torch.float32 or cos_sin.get_device() != index or cos_sin.dim() != 2 or
            cos_sin.shape[1] != D or not cos_sin.is_contiguous()):
        raise ValueError(f"cos_sin must be a contiguous fp32 tensor [max_pos, {D}] on cuda:{index}")
    if out is None:
        out, os = q.new_empty((M, Hq, D)), Hq * D
    else:
        os = _rows(out, "out", M, Hq, D, index)
        if M == 1 and out.data_ptr() == q.data_ptr():
            os = qs
    with _on(index):
        st = _b.lib().bitlinear_kv4_append(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, M, Hq,
                                           cos_sin.data_ptr(), cos_sin.shape[0], 1 if interleaved else 0, cache._c, batch,
                                           out.data_ptr(), os, _b._raw_stream(index))
    if st:
        _b._check(st, "bitlinear_kv4_append")
    return out


def kv4_read(cache: Kv4Cache, page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor, rows: int):
    """The cached values of the batch's tokens: (k, v), bf16 [rows, kv_heads, D]."""
    index = cache._index
    batch = _batch(index, page_table, kv_len, q_start)
    k = cache.k_steps.new_empty((rows, cache.kv_heads, cache.head_dim))
    v = torch.empty_like(k)
    with _on(index):
        st = _b.lib().bitlinear_kv4_read(cache._c, batch, rows, k.data_ptr(), v.data_ptr(), _b._raw_stream(index))
    if st:
        _b._check(st, "bitlinear_kv4_read")
    return k, v


def kv4_attention(q: torch.Tensor, cache: Kv4Cache, page_table: torch.Tensor, kv_len: torch.Tensor,
                  q_start: torch.Tensor, max_q: int, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of the batch's tokens q [M, Hq, D] bf16 over the cache (their own keys stored before):
    bf16 [M, Hq, D]. max_q: the largest number of new tokens of a sequence; scale: 1 / sqrt(D) by default."""
    D, index = cache.head_dim, cache._index
    M, Hq, _ = q.shape
    batch = _batch(index, page_table, kv_len, q_start)
    qs = _rows(q, "q", M, Hq, D, index)
    with _on(index):
        if out is None:
            out, os = q.new_empty((M, Hq, D)), Hq * D
        else:
            os = _rows(out, "out", M, Hq, D, index)
        if ws is None:
            need = _workspace_bytes(_b.BL_OP_KV4_ATTENTION, max_q, Hq // cache.kv_heads, D)
            ws = q.new_empty((need + 1) // 2)
        st = _b.lib().bitlinear_kv4_attention(q.data_ptr(), qs, M, Hq, max_q, D ** -0.5 if scale is None else scale,
                                              cache._c, batch, out.data_ptr(), os, ws.data_ptr(), ws.nbytes,
                                              _b._raw_stream(index))
    if st:
        _b._check(st, "bitlinear_kv4_attention")
    return out
