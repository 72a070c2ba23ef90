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

import ctypes
from contextlib import nullcontext
from typing import Optional

import torch

from . import binding as _b

GROUP = 32  # dims that share a quantisation step


class _CacheStruct(ctypes.Structure):
    _fields_ = [("kc", ctypes.c_void_p), ("ks", ctypes.c_void_p), ("vc", ctypes.c_void_p), ("vs", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("S", ctypes.c_int32), ("W", ctypes.c_int32)]


class Kv4Cache:
    """The four arrays of a cache: codes uint8 [num_pages, kv_heads, page_size, head_dim / 2] and
    steps bf16 [num_pages, kv_heads, page_size, head_dim / 32], of the keys and of the values."""

    __slots__ = ("k_codes", "k_steps", "v_codes", "v_steps", "_c")

    def __init__(self, k_codes: torch.Tensor, k_steps: torch.Tensor, v_codes: torch.Tensor, v_steps: torch.Tensor):
        if k_codes.dim() != 4:
            raise ValueError("codes must be [num_pages, kv_heads, page_size, head_dim / 2]")
        pages, heads, size, half = k_codes.shape
        for t, name, dtype, last in ((k_codes, "k_codes", torch.uint8, half), (v_codes, "v_codes", torch.uint8, half),
                                     (k_steps, "k_steps", torch.bfloat16, 2 * half // GROUP),
                                     (v_steps, "v_steps", torch.bfloat16, 2 * half // GROUP)):
            _b._cuda(t, name, dtype)
            if t.shape != (pages, heads, size, last) or t.device != k_codes.device:
                raise ValueError(f"{name} does not match k_codes {tuple(k_codes.shape)} on {k_codes.device}")
        self.k_codes, self.k_steps, self.v_codes, self.v_steps = k_codes, k_steps, v_codes, v_steps
        self._c = _CacheStruct(k_codes.data_ptr(), k_steps.data_ptr(), v_codes.data_ptr(), v_steps.data_ptr(),
                               pages, size, heads, 2 * half)


def kv4_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int, device) -> Kv4Cache:
    """An empty cache (zeroed)."""
    codes = (num_pages, kv_heads, page_size, head_dim // 2)
    steps = (num_pages, kv_heads, page_size, head_dim // GROUP)
    return Kv4Cache(torch.zeros(codes, dtype=torch.uint8, device=device),
                    torch.zeros(steps, dtype=torch.bfloat16, device=device),
                    torch.zeros(codes, dtype=torch.uint8, device=device),
                    torch.zeros(steps, dtype=torch.bfloat16, device=device))


def _on(device: torch.device):
    """The device of a call made current for it."""
    return nullcontext() if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _batch(cache: Kv4Cache, page_table, kv_len, q_start) -> _BatchStruct:
    dev = cache.k_codes.device
    for t, name in ((kv_len, "kv_len"), (q_start, "q_start"), (page_table, "page_table")):
        if t.dtype != torch.int32 or t.device != dev:
            raise ValueError(f"{name} must be an int32 tensor on {dev}")
    if page_table.dim() != 2 or page_table.stride(1) != 1 and page_table.shape[1] > 1:
        raise ValueError("page_table must be [S, W] with contiguous rows")
    S, W = page_table.shape
    if kv_len.shape != (S,) or q_start.shape != (S + 1,) or not kv_len.is_contiguous() or not q_start.is_contiguous():
        raise ValueError(f"kv_len must be [{S}] and q_start [{S + 1}], contiguous")
    return _BatchStruct(q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), page_table.stride(0), S, W)


def _rows(t: torch.Tensor, name: str, M: int, heads: Optional[int], D: int, device) -> int:
    """Row stride of t [M, heads, D] bf16 with the heads of a row side by side."""
    if t.dtype != torch.bfloat16 or t.device != device:
        raise ValueError(f"{name} must be a bf16 tensor on {device}")
    if t.dim() != 3 or t.shape[0] != M or t.shape[2] != D or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [{M}, {'heads' if heads is None else heads}, {D}], got {tuple(t.shape)}")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != D):
        raise ValueError(f"{name} must have the heads of a row side by side")
    return t.stride(0) if M > 1 else max(t.stride(0), t.shape[1] * D) // 8 * 8


def kv4_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos_sin: torch.Tensor, cache: Kv4Cache,
               page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor, interleaved: bool = False,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate q and k [M, heads, D] bf16 by their positions' rows of cos_sin [max_pos, D] fp32 (D/2 cosines, D/2 sines),
    store k and v in the cache and return the rotated q (in `out`, which may be q)."""
    c = cache._c
    dev, D = cache.k_codes.device, c.head_dim
    M, Hq = q.shape[0], q.shape[1]
    b = _batch(cache, page_table, kv_len, q_start)
    qs = _rows(q, "q", M, None, D, dev)
    ks = _rows(k, "k", M, c.kv_heads, D, dev)
    vs = _rows(v, "v", M, c.kv_heads, D, dev)
    _b._cuda(cos_sin, "cos_sin", torch.float32)
    if cos_sin.dim() != 2 or cos_sin.shape[1] != D or cos_sin.device != dev:
        raise ValueError(f"cos_sin must be [max_pos, {D}] on {dev}")
    if out is None:
        out = torch.empty((M, Hq, D), dtype=torch.bfloat16, device=dev)
    os = _rows(out, "out", M, Hq, D, dev)
    with _on(dev):
        st = _b.lib().bitlinear_kv4_append(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, M, Hq,
                                           cos_sin.data_ptr(), cos_sin.shape[0], int(bool(interleaved)),
                                           ctypes.byref(c), ctypes.byref(b), out.data_ptr(), os, _b._stream(dev))
    _b._check(st, "bitlinear_kv4_append")
    return out


def kv4_read(cache: Kv4Cache, page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor, rows: int):
    """The cached values of the batch's tokens: (k, v), bf16 [rows, kv_heads, D]."""
    c = cache._c
    dev = cache.k_codes.device
    b = _batch(cache, page_table, kv_len, q_start)
    k = torch.empty((rows, c.kv_heads, c.head_dim), dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    with _on(dev):
        st = _b.lib().bitlinear_kv4_read(ctypes.byref(c), ctypes.byref(b), rows, k.data_ptr(), v.data_ptr(),
                                         _b._stream(dev))
    _b._check(st, "bitlinear_kv4_read")
    return k, v


def kv4_attention(q: torch.Tensor, cache: Kv4Cache, page_table: torch.Tensor, kv_len: torch.Tensor,
                  q_start: torch.Tensor, max_q: int, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of the batch's tokens q [M, Hq, D] bf16 over the cache (their own keys stored before):
    bf16 [M, Hq, D]. max_q: the largest number of new tokens of a sequence; scale: 1 / sqrt(D) by default."""
    c = cache._c
    dev, D = cache.k_codes.device, c.head_dim
    M, Hq = q.shape[0], q.shape[1]
    b = _batch(cache, page_table, kv_len, q_start)
    qs = _rows(q, "q", M, None, D, dev)
    if out is None:
        out = torch.empty((M, Hq, D), dtype=torch.bfloat16, device=dev)
    os = _rows(out, "out", M, Hq, D, dev)
    with _on(dev):
        if ws is None:
            ws = torch.empty(_b.workspace_bytes(_b.BL_OP_KV4_ATTENTION, max_q, Hq // c.kv_heads, D), dtype=torch.uint8, device=dev)
        st = _b.lib().bitlinear_kv4_attention(q.data_ptr(), qs, M, Hq, int(max_q), D ** -0.5 if scale is None else scale,
                                              ctypes.byref(c), ctypes.byref(b), out.data_ptr(), os, ws.data_ptr(),
                                              ws.numel(), _b._stream(dev))
    _b._check(st, "bitlinear_kv4_attention")
    return out
