"""One decoder block of a BitNet b1.58 model on the library's calls: Q/K/V in one
projection after the pre-norm, rotation and 4-bit cache, attention, the output
projection after its subln with the residual, the FFN with its residual.

The paper card "BitNet b1.58 2B4T Technical Report", "Method Adaptation", names the
parts (BitLinear in place of the linear layers, subln, ReLU^2, rotary positions); this
module only puts the calls in order and computes nothing itself.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import binding as _b
from . import kv4 as _kv4


@dataclass
class Block:
    """Packed weights of a block, as pack_weights gives them; the Q, K and V rows stacked."""
    Wqkv: torch.Tensor  # [(Hq + 2 Hkv) D, d / 4]
    gqkv: torch.Tensor  # [3]: gammas of Q, K and V
    Wo: torch.Tensor    # [d, Hq D / 4]
    go: torch.Tensor    # [1]
    Wg: torch.Tensor    # [f, d / 4]
    gg: torch.Tensor
    Wu: torch.Tensor
    gu: torch.Tensor
    Wd: torch.Tensor    # [d, f / 4]
    gd: torch.Tensor

    @classmethod
    def pack(cls, Wq, Wk, Wv, Wo, Wg, Wu, Wd) -> "Block":
        """From the bf16 or fp32 weights."""
        qkv = [_b.pack_weights(w) for w in (Wq, Wk, Wv)]
        rest = [t for w in (Wo, Wg, Wu, Wd) for t in _b.pack_weights(w)]
        return cls(torch.cat([w for w, _ in qkv]), torch.cat([g.reshape(1) for _, g in qkv]), *rest)


def decoder_block(block: Block, h: torch.Tensor, heads: int, cache: _kv4.Kv4Cache, cos_sin: torch.Tensor,
                  page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor, max_q: int,
                  scale: Optional[float] = None, interleaved: bool = False) -> torch.Tensor:
    """h [M, d] bf16 (the batch's new tokens) -> the block's output [M, d]; keys and values go to `cache`, which is the
    block's own. `heads`: query heads; the batch and `max_q` as in kv4_attention."""
    D, hkv = cache.head_dim, cache.kv_heads
    rows = [heads * D, hkv * D, hkv * D]
    qkv = _b.forward_ex(block.Wqkv, block.gqkv, rows, h, rmsnorm=True, ws=_scratch(_b.BL_OP_FORWARD, h, sum(rows)))
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split(rows, 1))
    # in place: padding rows of a batch keep finite values that way
    q = _kv4.kv4_append(q, k, v, cos_sin, cache, page_table, kv_len, q_start, interleaved, out=q)
    o = torch.zeros((h.shape[0], heads * D), dtype=torch.bfloat16, device=h.device)
    _kv4.kv4_attention(q, cache, page_table, kv_len, q_start, max_q, scale, out=o.unflatten(1, (heads, D)))
    h = _b.forward_ex(block.Wo, block.go, [block.Wo.shape[0]], o, rmsnorm=True, residual=h,
                      ws=_scratch(_b.BL_OP_FORWARD, o, block.Wo.shape[0]))
    return _b.ffn(block.Wg, block.gg, block.Wu, block.gu, block.Wd, block.gd, h, residual=h,
                  ws=_scratch(_b.BL_OP_FFN, h, block.Wg.shape[0]))


def _scratch(op: int, x: torch.Tensor, N: int) -> torch.Tensor:
    """Scratch of one call: blocks on different streams, or in captured graphs, share none."""
    return torch.empty(_b.workspace_bytes(op, x.shape[0], N, x.shape[1]), dtype=torch.uint8, device=x.device)
