"""Norms and the block quantizer in every number of pieces that a thread may hold of a row, in all their outputs, with ends of rows inside
a wave's run.  Tolerances: test_gpu_norm.py's; the quantizer's codes and scales are equal."""
import numpy as np
import pytest
import torch

import plain_layer as plain
from parity import say
from test_gpu_fp8_block import act_codes
from test_gpu_fp8_block import inputs as product_inputs
from test_gpu_norm import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


# up to 1 piece of 8 columns in 1,024 threads, 2, 3, 4, 8 and 16, and for 257 rows and more in 512
@pytest.mark.parametrize("M,K", ((3, 8192), (3, 8320), (3, 16384), (3, 18560), (5, 24576), (3, 24704), (2, 32768), (3, 32896), (2, 65536), (2, 65664),
                                 (259, 4096), (259, 4224), (300, 8320), (300, 13440), (259, 16384), (259, 16512)))
def test_quantizer(lib, M, K):
    say(f"block quantizer {M} x {K}")
    x, _, _ = product_inputs(M, 8, K, M + K)
    q, s = act_codes(x)
    gq, gs = lib.w8a8_quantize_act_block(x.cuda())
    assert np.array_equal(gq.cpu().numpy(), q) and np.array_equal(gs.cpu().numpy(), s)
    pq, ps = lib.w8a8_quantize_act_block_packed(x.cuda())
    assert np.array_equal(plain.unpack(pq.cpu().numpy(), M, K), q) and np.array_equal(ps.cpu().numpy()[:, :M].T, s)


@pytest.mark.parametrize("M,K", ((3, 8192), (3, 8320), (3, 16512), (3, 24704), (2, 32768), (3, 32896), (2, 65536), (2, 65664),
                                 (259, 4224), (259, 8320), (259, 13440), (259, 16512)))
@pytest.mark.parametrize("form,rot", (("bf16", 0), ("int8", 0), ("int8", 128), ("fp8", 0), ("fp8", 128), ("block", 0)))
def test_norm(lib, M, K, form, rot):
    say(f"norm {M} x {K} {form}, rotated {rot}")
    x, res, w = inputs(M, K, M + K)
    check(lib, x, res, w, 1e-6, form, rot)
    check(lib, x, None, w, 1e-6, form, rot, packed=form != "bf16")
