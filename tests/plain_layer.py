"""Plain 64-bit forms of the operators around the projections, from their formulas (numpy and torch on the CPU): norms,
rotary positions, E4M3 projections with block scales.

They share nothing with the kernels.  Codes round as the formulas do (single fp32 divisions, nearest even); everything else
is fp64.
"""
import math

import numpy as np
import torch

F8_MAX = np.float32(448)


def bf16(a):
    """numpy -> the nearest bf16 values, as a torch tensor."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def hadamard():
    """The normalized Sylvester matrix of order 128."""
    i = np.arange(128)
    return (1.0 - 2.0 * (np.vectorize(lambda v: bin(v).count("1"))(i[:, None] & i) % 2)) / math.sqrt(128)


def int8_codes(v, s):
    """v fp32 [rows, n], s fp32 [rows]: nearest-even codes of the fp32 quotients; zeros where s is zero."""
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(v / s[:, None])
    return np.where(s[:, None] > 0, q, 0).astype(np.int8)


def e4m3_codes(v, s):
    """v fp32 [rows, n], s fp32 [rows] -> E4M3FN codes of clamp(v / s, +-448); +0 where s is zero."""
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.clip(v / s[:, None], -F8_MAX, F8_MAX)
    codes = torch.from_numpy(np.where(s[:, None] > 0, q, 0).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return np.where(s[:, None] > 0, codes, 0).astype(np.uint8)


def e4m3_values(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def unpack(packed, rows, K):
    """Row-major bytes [rows, K] of the packed layout, address by address."""
    r, k = np.arange(rows)[:, None], np.arange(K)
    return np.asarray(packed)[(r // 32 * (K // 64) + k // 64) * 2048 + r % 32 * 64 + k % 64]


def pack(codes):
    """The packed layout of row-major bytes, padding rows zero."""
    rows, K = codes.shape
    out = np.zeros(-(-rows // 32) * 32 * K, dtype=np.uint8)
    r, k = np.arange(rows)[:, None], np.arange(K)
    out[(r // 32 * (K // 64) + k // 64) * 2048 + r % 32 * 64 + k % 64] = codes.view(np.uint8)
    return out


def norm(x, residual, weight, eps):
    """(y, z, r, h): y = z * r fp64, z = h * weight, r [rows, 1], h the bf16 sum (fp32 addition, rounded) as fp64."""
    h = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    v = f64(h)
    z = v * f64(weight)
    r = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return z * r, z, r, h


def turned(x, lens, turns, interleaved, amplitude):
    """(y, spread): the rotation of x [seqs, tokens, heads, dim] by exact fractions of a turn, and |a| + |b| of each value's pair."""
    seqs, tokens, _, _ = x.shape
    half = len(turns)
    first, second = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if interleaved else (np.arange(half), np.arange(half, 2 * half))
    y, spread = x.copy(), np.zeros_like(x)
    for b in range(seqs):
        for t in range(tokens):
            p = max(int(lens[b]), 0) - tokens + t
            if p < 0:
                continue
            angle = np.array([2 * math.pi * ((p * int(f)) % (1 << 64) / 2.0 ** 64) for f in turns])
            u, v = x[b, t][:, first], x[b, t][:, second]
            y[b, t][:, first] = amplitude * (u * np.cos(angle) - v * np.sin(angle))
            y[b, t][:, second] = amplitude * (v * np.cos(angle) + u * np.sin(angle))
            spread[b, t][:, first] = spread[b, t][:, second] = np.abs(amplitude) * (np.abs(u) + np.abs(v))
    return y, spread


def block_product(q, s, w, sw, bias):
    """(y, dropped, spread) fp64 [M, N] of codes q [M, K], w [N, K] with scales s [M, K / 128], sw [ceil(N / 128), K / 128]:
    the sum; the most that the matrix instruction may drop of it (each product what lies 2^-13 below the largest of its block);
    and the sum of the products' magnitudes."""
    a, b = e4m3_values(q), e4m3_values(w)
    M, N, K = a.shape[0], b.shape[0], a.shape[1]
    y, dropped, spread = (np.zeros((M, N)) for _ in range(3))
    for i in range(K // 128):
        x, v = a[:, 128 * i:128 * i + 128], b[:, 128 * i:128 * i + 128]
        by = s[:, i].astype(np.float64)[:, None] * np.repeat(sw[:, i].astype(np.float64), 128)[None, :N]
        p = np.abs(x[:, None, :] * v[None, :, :])
        y += (x @ v.T) * by
        dropped += np.minimum(p, p.max(-1, keepdims=True) * 2.0 ** -13).sum(-1) * by
        spread += p.sum(-1) * by
    if bias is not None:
        y, spread = y + f64(bias), spread + np.abs(f64(bias))
    return y, dropped, spread
