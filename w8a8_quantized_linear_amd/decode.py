"""One decoder layer that answers: the prompt through the 8-bit projections, then tokens one at a time through
the 4-bit ones, with the paged 8-bit cache and its attention between them.

What it computes, for x [seqs, tokens, hidden] (the newest tokens of each sequence):

    q, k, v = norm1(x) Wqkv^T     q, k = rotate(q, k); k and v appended to the cache, q attends to it
    x = x + attention Wo^T
    h = norm2(x)
    x = x + (silu(h Wgate^T) * (h Wup^T)) Wdown^T

Norms and the rotation of q and k by position are functions that the caller gives (they are elementwise and not part
of this library); without them the layer leaves them out.  Each weight is held twice: int8 for calls of many tokens (one GEMM serves all of them), and
4-bit codes for calls of few, which are bound by the weights' bytes.  Nothing below synchronizes or reads
device memory on the host, so a step may be captured into a HIP graph and replayed while `lens` grows.

``python bench.py --decode`` runs it: a prompt, then a captured step.
"""
from __future__ import annotations

from typing import Callable, Optional, Tuple

import torch

from . import (KVCache, w8a8_gateup_swiglu_packed, w8a8_kv_append, w8a8_kv_attention, w8a8_linear_packed,
               w8a8_pack_weight, w8a8_quantize_act, w8a8_swiglu, w8a8_w4_linear, w8a8_w4_pack, w8a8_w4_quantize)


class Projection:
    """y = x W^T for W bf16 [N, K] in both forms; `few` tokens and fewer take the 4-bit one.

    Where the forms cross depends on the shape: 64 tokens take 14 us in 4 bits and 26 us in 8 for 5,120 x 7,168,
    31 and 69 us for 17,408 x 5,120, but 49 and 37 us for 5,120 x 34,816, and 32 tokens 30 and 36 us there."""

    def __init__(self, w: torch.Tensor, group: int, few: int):
        self.N, self.group, self.few = w.shape[0], group, few
        codes, self.s8 = w8a8_quantize_act(w)
        self.w8 = w8a8_pack_weight(codes)
        self.w4 = w8a8_w4_pack(*w8a8_w4_quantize(w, group))

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[0] <= self.few:
            return w8a8_w4_linear(x, *self.w4, self.N, self.group)
        return w8a8_linear_packed(x, self.w8, self.N, self.s8)


class DecoderLayer:
    """wqkv bf16 [(q_heads + 2 heads) * dim, hidden], wo [hidden, q_heads * dim], wgateup [2 ffn, hidden],
    wdown [hidden, ffn]; calls of up to `few` tokens in all sequences use 4-bit weights in groups of `group`.
    norm1 and norm2: bf16 [tokens, hidden] -> the same, before the attention and before the MLP."""

    def __init__(self, wqkv, wo, wgateup, wdown, q_heads: int, heads: int, dim: int, group: int = 64, few: int = 32,
                 norm1: Optional[Callable[[torch.Tensor], torch.Tensor]] = None,
                 norm2: Optional[Callable[[torch.Tensor], torch.Tensor]] = None):
        self.norm1, self.norm2 = norm1, norm2
        self.q_heads, self.heads, self.dim, self.ffn = q_heads, heads, dim, wdown.shape[1]
        if wqkv.shape[0] != (q_heads + 2 * heads) * dim or wo.shape[1] != q_heads * dim or wgateup.shape[0] != 2 * self.ffn:
            raise ValueError("weights and head counts disagree")
        self.qkv, self.o, self.gateup, self.down = (Projection(w, group, few) for w in (wqkv, wo, wgateup, wdown))

    def __call__(self, x: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                 scale: Optional[float] = None,
                 rotate: Optional[Callable[[torch.Tensor, torch.Tensor], Tuple[torch.Tensor, torch.Tensor]]] = None) -> torch.Tensor:
        """x bf16 [seqs, tokens, hidden] -> the same shape; lens counts these tokens already.  rotate: (q, k), bf16
        [seqs, tokens, heads, dim] each, at positions lens - tokens .. lens - 1 -> the same, rotated."""
        seqs, tokens, hidden = x.shape
        rows = x.reshape(seqs * tokens, hidden)
        qkv = self.qkv(rows if self.norm1 is None else self.norm1(rows)).view(seqs, tokens, self.q_heads + 2 * self.heads, self.dim)
        q, k, v = qkv.split((self.q_heads, self.heads, self.heads), dim=2)      # slices: none is copied
        if rotate is not None:
            q, k = rotate(q, k)
        w8a8_kv_append(k, v, cache, table, lens)
        a = w8a8_kv_attention(q, cache, table, lens, scale)
        rows = rows + self.o(a.view(seqs * tokens, self.q_heads * self.dim))
        h = rows if self.norm2 is None else self.norm2(rows)
        if rows.shape[0] <= self.gateup.few:
            h = self.gateup(h)
            h = w8a8_swiglu(h[:, :self.ffn], h[:, self.ffn:])
        else:
            h = w8a8_gateup_swiglu_packed(h, self.gateup.w8, self.ffn, self.gateup.s8)
        return (rows + self.down(h)).view(seqs, tokens, hidden)


def random_layer(hidden: int, q_heads: int, heads: int, dim: int, ffn: int, group: int = 64, few: int = 32, seed: int = 0,
                 device="cuda") -> DecoderLayer:
    """A layer with normal weights of 1 / sqrt(K), drawn on the device."""
    g = torch.Generator(device=device).manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g, device=device, dtype=torch.bfloat16) * k ** -0.5)
    return DecoderLayer(w((q_heads + 2 * heads) * dim, hidden), w(hidden, q_heads * dim), w(2 * ffn, hidden), w(hidden, ffn),
                        q_heads, heads, dim, group, few)
