"""Attention of long sequences: at the end of the running sum's range."""
import numpy as np
import pytest
import torch

from parity import say
from test_gpu_kv_attention import attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def test_the_sum_over_a_long_sequence_of_small_values(lib):
    """2^24 tokens whose values have the smallest scale that counts, 2^-90, and whose scores lie 7.9 powers of two above
    the first ones, which the running maximum does not follow: the sum of p / scale passes 2^128.  All tokens but the
    first page's share one page, so the cache is small; 512 heads, so the sequence is one piece.

    y is 100 * 2^-90 but for the first page's 128 tokens (2^-17 of it): fp32 sums of 2^17 equal steps in a row err by up
    to 2^-8 each, outputs and sum, and bf16 by 2^-9, so within 2^-6."""
    heads, dim, page, length = 512, 64, 128, 1 << 24
    say("2^24 tokens of 512 heads")
    cache = lib.kv_cache(2, heads, page, dim)
    for t in cache[:2]:
        t.zero_()
    cache.k_codes[1, :, :, 0] = 79
    cache.v_codes[0], cache.v_codes[1] = 10, 100
    cache.k_scale.fill_(7.9 / 79 * float(np.log(2)))
    cache.v_scale.fill_(2.0 ** -90)
    table = torch.ones(1, length // page, dtype=torch.int32)
    table[0, 0] = 0
    assert lib.kv_attention_workspace_bytes(1, 1, heads, heads, dim, page, table.shape[1]) == 0
    q = torch.zeros(1, 1, heads, dim, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    y = attend(lib, q, cache, table, [length], 1.0).double().cpu() * 2.0 ** 90
    assert float((y / 100 - 1).abs().max()) < 2 ** -6, y.flatten()[:4]
