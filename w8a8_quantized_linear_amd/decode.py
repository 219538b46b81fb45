"""One decoder layer that answers: the prompt through the 8-bit projections, then tokens one at a time through
the 4-bit ones, with the paged 8-bit cache and its attention between them; or all of it through E4M3 projections with
block scales.

What it computes, for x [seqs, tokens, hidden] (the newest tokens of each sequence):

    q, k, v = norm1(x) Wqkv^T     q, k = rotate(q, k); k and v appended to the cache, q attends to it
    x = x + attention Wo^T
    h = norm2(x)
    x = x + (silu(h Wgate^T) * (h Wup^T)) Wdown^T

norm1 and norm2 are weights of root-mean-square norms (bf16 [hidden]), or functions that the caller gives; rotate is a plan
of rotary positions (``Rope``), or a function; without them the layer leaves them out.  With weights, a norm adds the
residual and quantizes for the projection behind it in one launch, and so does the norm of the next layer where layers
are chained by ``step``.

Projections hold each weight twice (``Projection``): int8 for calls of many tokens (one GEMM serves all of them), and 4-bit
codes for calls of few, which are bound by the weights' bytes; or once (``BlockProjection``): E4M3 codes with a scale for each
128 x 128 block, for any number of tokens.  Nothing below synchronizes or reads device memory on the host, so a step may
be captured into a HIP graph and replayed while `lens` grows.

``python bench.py --decode`` runs it: a prompt, then a captured step.
"""
from __future__ import annotations

from typing import Callable, Optional, Tuple, Union

import torch

from . import (KVCache, Rope, w8a8_fp8_block_gemm_packed, w8a8_fp8_block_linear_packed, w8a8_gateup_swiglu_packed,
               w8a8_gemm_dequant_packed, w8a8_gemm_swiglu_packed, w8a8_kv_append, w8a8_kv_attention, w8a8_linear_packed,
               w8a8_pack_weight, w8a8_quantize_act, w8a8_quantize_weight_block, w8a8_rmsnorm, w8a8_rmsnorm_quantize_block_packed,
               w8a8_rmsnorm_quantize_packed, w8a8_rope, w8a8_swiglu, w8a8_w4_linear, w8a8_w4_pack, w8a8_w4_quantize)


class Projection:
    """y = x W^T for W bf16 [N, K] in both forms; `few` tokens and fewer take the 4-bit one.

    Where the forms cross depends on the shape: 64 tokens take 14 us in 4 bits and 26 us in 8 for 5,120 x 7,168,
    31 and 69 us for 17,408 x 5,120, but 49 and 37 us for 5,120 x 34,816, and 32 tokens 30 and 36 us there."""

    def __init__(self, w: torch.Tensor, group: int, few: int):
        (self.N, self.K), self.group, self.few = w.shape, group, few
        codes, self.s8 = w8a8_quantize_act(w)
        self.w8 = w8a8_pack_weight(codes)
        self.w4 = w8a8_w4_pack(*w8a8_w4_quantize(w, group))

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[0] <= self.few:
            return w8a8_w4_linear(x, *self.w4, self.N, self.group)
        return w8a8_linear_packed(x, self.w8, self.N, self.s8)

    def behind_norm(self, x, weight, eps, residual):
        """(norm(x + residual) W^T, x + residual); the norm quantizes for the 8-bit form."""
        if x.shape[0] <= self.few:
            y, h = w8a8_rmsnorm(x, weight, residual, eps)
            return self(y), x if h is None else h
        q, s, h = w8a8_rmsnorm_quantize_packed(x, weight, residual, eps)
        return w8a8_gemm_dequant_packed(q, s, self.w8, self.s8, self.K), x if h is None else h

    def swiglu(self, x: torch.Tensor) -> torch.Tensor:
        """silu(x Wgate^T) * (x Wup^T) for W = [Wgate; Wup]."""
        if x.shape[0] <= self.few:
            return _swiglu(self(x))
        return w8a8_gateup_swiglu_packed(x, self.w8, self.N // 2, self.s8)

    def swiglu_behind_norm(self, x, weight, eps, residual):
        if x.shape[0] <= self.few:
            y, h = self.behind_norm(x, weight, eps, residual)
            return _swiglu(y), h
        q, s, h = w8a8_rmsnorm_quantize_packed(x, weight, residual, eps)
        return w8a8_gemm_swiglu_packed(q, s, self.w8, self.s8, self.K), x if h is None else h


class BlockProjection:
    """y = x W^T for W bf16 [N, K] as E4M3 codes with a scale for each 128 x 128 block."""

    def __init__(self, w: torch.Tensor):
        self.N, self.K = w.shape
        codes, self.s = w8a8_quantize_weight_block(w)
        self.w = w8a8_pack_weight(codes)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return w8a8_fp8_block_linear_packed(x, self.w, self.N, self.s)

    def behind_norm(self, x, weight, eps, residual):
        q, s, h = w8a8_rmsnorm_quantize_block_packed(x, weight, residual, eps)
        return w8a8_fp8_block_gemm_packed(q, s, self.w, self.s, x.shape[0], self.N, self.K), x if h is None else h

    def swiglu(self, x: torch.Tensor) -> torch.Tensor:
        return _swiglu(self(x))

    def swiglu_behind_norm(self, x, weight, eps, residual):
        y, h = self.behind_norm(x, weight, eps, residual)
        return _swiglu(y), h


def _swiglu(gateup: torch.Tensor) -> torch.Tensor:
    half = gateup.shape[1] // 2
    return w8a8_swiglu(gateup[:, :half], gateup[:, half:])


Norm = Union[torch.Tensor, Callable[[torch.Tensor], torch.Tensor], None]
Rotation = Union[Rope, Callable[[torch.Tensor, torch.Tensor], Tuple[torch.Tensor, torch.Tensor]], None]


class DecoderLayer:
    """wqkv bf16 [(q_heads + 2 heads) * dim, hidden], wo [hidden, q_heads * dim], wgateup [2 ffn, hidden],
    wdown [hidden, ffn]; calls of up to `few` tokens in all sequences use 4-bit weights in groups of `group`; blocks: E4M3
    projections with block scales instead.
    norm1 and norm2, before the attention and before the MLP: weights bf16 [hidden] of root-mean-square norms with `eps`, or
    functions, bf16 [tokens, hidden] -> the same."""

    def __init__(self, wqkv, wo, wgateup, wdown, q_heads: int, heads: int, dim: int, group: int = 64, few: int = 32,
                 norm1: Norm = None, norm2: Norm = None, eps: float = 1e-6, blocks: bool = False):
        self.norm1, self.norm2, self.eps = norm1, norm2, eps
        self.q_heads, self.heads, self.dim, self.ffn = q_heads, heads, dim, wdown.shape[1]
        if wqkv.shape[0] != (q_heads + 2 * heads) * dim or wo.shape[1] != q_heads * dim or wgateup.shape[0] != 2 * self.ffn:
            raise ValueError("weights and head counts disagree")
        self.qkv, self.o, self.gateup, self.down = (BlockProjection(w) if blocks else Projection(w, group, few)
                                                    for w in (wqkv, wo, wgateup, wdown))

    def step(self, x: torch.Tensor, residual: Optional[torch.Tensor], cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
             scale: Optional[float] = None, rotate: Rotation = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """What the layer adds, and what it adds it to: (y, residual), bf16 [seqs, tokens, hidden] each, whose sum is the layer's
        output; it takes its input as such a pair too (residual None: x alone), so that the sums are left to the norms."""
        seqs, tokens, hidden = x.shape
        rows = x.contiguous().view(seqs * tokens, hidden)                       # (copied where it is a slice: the last tokens of prompts)
        before = None if residual is None else residual.contiguous().view(seqs * tokens, hidden)
        if isinstance(self.norm1, torch.Tensor):
            qkv, rows = self.qkv.behind_norm(rows, self.norm1, self.eps, before)
        else:
            rows = rows if before is None else rows + before
            qkv = self.qkv(rows if self.norm1 is None else self.norm1(rows))
        q, k, v = qkv.view(seqs, tokens, self.q_heads + 2 * self.heads, self.dim).split((self.q_heads, self.heads, self.heads), dim=2)
        if isinstance(rotate, Rope):                                            # (slices: none is copied)
            q, k = w8a8_rope(q, k, lens, rotate, out=(q, k))
        elif rotate is not None:
            q, k = rotate(q, k)
        w8a8_kv_append(k, v, cache, table, lens)
        a = self.o(w8a8_kv_attention(q, cache, table, lens, scale).view(seqs * tokens, self.q_heads * self.dim))
        if isinstance(self.norm2, torch.Tensor):
            h, rows = self.gateup.swiglu_behind_norm(a, self.norm2, self.eps, rows)
        else:
            rows = rows + a
            h = self.gateup.swiglu(rows if self.norm2 is None else self.norm2(rows))
        return self.down(h).view(seqs, tokens, hidden), rows.view(seqs, tokens, hidden)

    def __call__(self, x: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                 scale: Optional[float] = None, rotate: Rotation = None) -> torch.Tensor:
        """x bf16 [seqs, tokens, hidden] -> the same shape; lens counts these tokens already.  rotate: a plan of rotary positions
        (``rope``), or a function: (q, k), bf16 [seqs, tokens, heads, dim] each, at positions lens - tokens .. lens - 1 -> the same,
        rotated."""
        y, rows = self.step(x, None, cache, table, lens, scale, rotate)
        return rows + y


def random_layer(hidden: int, q_heads: int, heads: int, dim: int, ffn: int, group: int = 64, few: int = 32, seed: int = 0,
                 device="cuda", norms: bool = False, blocks: bool = False) -> DecoderLayer:
    """A layer with normal weights of 1 / sqrt(K), drawn on the device; norms: with root-mean-square norms, weights around 1."""
    g = torch.Generator(device=device).manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g, device=device, dtype=torch.bfloat16) * k ** -0.5)
    ws = w((q_heads + 2 * heads) * dim, hidden), w(hidden, q_heads * dim), w(2 * ffn, hidden), w(hidden, ffn)
    n1, n2 = ((1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(torch.bfloat16) if norms else None for _ in range(2))
    return DecoderLayer(*ws, q_heads, heads, dim, group, few, n1, n2, blocks=blocks)
