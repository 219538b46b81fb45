"""Norms of rows whose products h * weight leave fp32's normal range.

u = 2^-149, fp32's smallest step.  z rounds to a multiple of u: off by d = u / 2 (rotated: 128 of them over sqrt(128) and the
product's own: 6.2 u, and what test_gpu_norm.py allows for the butterflies).  Its scale, (amax / top), top 127 or 448, is off by u / 2 at
most, so a code's value is off by half its step or, where the quotient passes the largest code, by what that lacks of amax, top * u / 2.
Times r; and the stored scale rounds once more: top * u / 2.  Half a step: amax / 254 (+ u / 4, + d / 254: below another d); E4M3
2^-4 of the value, amax / 448 * 2^-10 at least."""
import numpy as np
import pytest
import torch

import plain_layer as plain
from parity import say
from test_gpu_norm import R_TOL, ROT_TOL

pytestmark = pytest.mark.gpu

U = 2.0 ** -149


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


@pytest.mark.parametrize("K", (128, 1152))
@pytest.mark.parametrize("form,rot", (("int8", 0), ("int8", 128), ("fp8", 0), ("fp8", 128), ("block", 0)))
def test_products_below_the_normal_range(lib, K, form, rot):
    """Rows of 2^-133 to 2^-120 by weights around 2^-1 to 2^-12: every value near its formula's."""
    say(f"norm of {K} small columns, {form}, rotated {rot}")
    rng = np.random.default_rng(K)
    h = rng.choice([-1.0, 1.0], (40, K)) * np.exp2(-133.0 + np.arange(40) % 14)[:, None] * rng.integers(1, 4, (40, K))
    w = 190 * np.exp2(rng.choice([-16.0, -17.0, -20.0], K))
    w[5] = 190 * 2.0 ** -16
    if K > 128:
        w[:256] *= 2.0 ** 7
    x, w = plain.bf16(h), plain.bf16(w)
    assert (plain.f64(x) == h).all()
    y, z, r, _ = plain.norm(x, None, w, 1e-6)
    top = 127.0 if form == "int8" else 448.0
    of = 128 if form == "block" else K
    name = {"int8": "w8a8_rmsnorm_quantize", "fp8": "w8a8_rmsnorm_quantize_fp8", "block": "w8a8_rmsnorm_quantize_block"}[form]
    q, s, _ = getattr(lib, name)(x.cuda(), w.cuda(), eps=1e-6, **({} if form == "block" else dict(rot_block=rot)))
    q, s = q.cpu().numpy(), s.cpu().numpy().astype(np.float64).reshape(40, -1)
    values = (q.astype(np.float64) if form == "int8" else plain.e4m3_values(q)) * np.repeat(s, of, axis=1)
    slack = 0.0
    if rot:
        slack = np.repeat(np.abs(y).reshape(40, -1, 128).sum(-1), 128, axis=1) * ROT_TOL / 128 ** 0.5
        y, z = ((v.reshape(-1, 128) @ plain.hadamard()).reshape(40, K) for v in (y, z))
    amax = np.repeat(np.abs(z).reshape(40, -1, of).max(-1), of, axis=1)
    step = amax / top if form == "int8" else np.maximum(np.abs(z) * 2.0 ** -3, amax / top * 2.0 ** -9)
    by = r * (np.maximum(step / 2, top * U / 2) + 2 * (6.2 if rot else 0.5) * U) + top * U / 2 + slack + np.abs(y) * R_TOL
    off = np.abs(values - y)
    assert (off <= by).all(), f"off by {np.max(off / by)} of what it may be"
