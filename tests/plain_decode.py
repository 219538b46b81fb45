"""Plain 64-bit forms of the few-token operators, from their formulas (numpy, CPU).

They share nothing with the kernels: no packed layout beyond the one documented in
``include/w8a8.h`` (read address by address), loops over sequences and heads, fp64 throughout
except where the formula itself rounds (codes and scales).
"""
import numpy as np


def w4_codes(codes, K):
    """Row-major bytes [N, K / 2] -> int codes [N, K] in [-8, 7]."""
    out = np.empty((codes.shape[0], K), dtype=np.int64)
    out[:, 0::2] = codes & 15
    out[:, 1::2] = codes >> 4
    return out - 8


def w4_linear(x, codes, scales, group, bias):
    """fp64 [M, N]; x [M, K], codes [N, K] ints, scales [N, K / group]."""
    w = codes.astype(np.float64) * np.repeat(scales.astype(np.float64), group, axis=1)
    y = x.astype(np.float64) @ w.T
    return y if bias is None else y + bias.astype(np.float64)


def w4_packed_byte(n, c, K):
    """(byte, shift) of column c of row n in the packed codes."""
    block = (n // 16) * (K // 128) + c // 128
    c, r, j = c % 128, n % 16, c % 8
    bit = 4 * (j // 2) + 16 * (j % 2)
    return block * 1024 + (16 * (c // 8 % 4) + r) * 16 + 4 * (c // 32) + bit // 8, bit % 8


def append(new, codes, scale, table, lens):
    """The cache's codes [pages, heads, page, dim] and scales [pages, heads] (changed in place) after the tokens
    `new` [seqs, tokens, heads, dim]: single fp32 operations where the formula has them (numpy's are IEEE)."""
    seqs, tokens, heads, dim = new.shape
    pages, page = codes.shape[0], codes.shape[2]
    new = new.astype(np.float32)
    for b in range(seqs):
        length = max(int(lens[b]), 0)
        held = min(length, table.shape[1] * page)
        for block in range(table.shape[1]):
            lo, hi = max(block * page, length - tokens, 0), min((block + 1) * page, held)
            p = int(table[b, block])
            if lo >= hi or not 0 <= p < pages:
                continue
            for h in range(heads):
                x = new[b, lo - (length - tokens):hi - (length - tokens), h]
                s_old = scale[p, h] if lo > block * page else np.float32(0)
                s = max(np.float32(s_old), np.abs(x).max() / np.float32(127))
                old = codes[p, h, :lo - block * page]
                if old.size and s > s_old:
                    ratio = np.float32(s_old) / s
                    codes[p, h, :lo - block * page] = np.rint(old.astype(np.float32) * ratio).astype(np.int8)
                q = np.rint(x / s) if s > 0 else np.zeros_like(x)
                codes[p, h, lo - block * page:hi - block * page] = q.astype(np.int8)
                scale[p, h] = s


def gathered(codes, scale, table, length, head):
    """fp64 values [length, dim] of one sequence and head, and which positions have a page."""
    pages, _, page, dim = codes.shape
    x, real = np.zeros((length, dim)), np.zeros(length, dtype=bool)
    for pos in range(0, length, page):
        p = int(table[pos // page])
        if 0 <= p < pages:
            n = min(page, length - pos)
            x[pos:pos + n] = codes[p, head, :n].astype(np.float64) * float(scale[p, head])
            real[pos:pos + n] = True
    return x, real


def attention(q, k_codes, v_codes, k_scale, v_scale, table, lens, scale):
    """(y, spread) fp64 [seqs, tokens, q_heads, dim]: the output and sum(p |v|) / sum(p), what a relative
    error of each probability is measured against."""
    seqs, tokens, q_heads, dim = q.shape
    heads, page = k_codes.shape[1], k_codes.shape[2]
    group = q_heads // heads
    y, spread = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(seqs):
        length = max(int(lens[b]), 0)
        held = min(length, table.shape[1] * page)
        for h in range(heads):
            k, real = gathered(k_codes, k_scale, table[b], held, h)
            v, _ = gathered(v_codes, v_scale, table[b], held, h)
            for i in range(tokens):
                seen = real & (np.arange(held) <= length - tokens + i)
                if not seen.any():
                    continue
                for a in range(h * group, (h + 1) * group):
                    s = scale * (k[seen] @ q[b, i, a].astype(np.float64))
                    p = np.exp(s - s.max())
                    y[b, i, a] = p @ v[seen] / p.sum()
                    spread[b, i, a] = p @ np.abs(v[seen]) / p.sum()
    return y, spread
