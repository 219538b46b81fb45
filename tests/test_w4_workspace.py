"""Workspace of the 4-bit projections where K is cut: bounded whatever the number of tokens (sizes on the CPU), and
calls of more tokens than one block of it serves."""
import pytest
import torch

from parity import say
from test_decode_abi import lib as abi      # noqa: F401  (the C library, as a fixture)
from test_gpu_w4 import run


def test_workspace_does_not_grow_past_a_block_of_tokens(abi):      # noqa: F811
    size = abi.w8a8_w4_workspace_bytes
    one = size(1, 5120, 17408)
    assert 0 < one <= 3 * 5120 * 4 + 255 and size(64, 5120, 17408) <= 64 * 3 * 5120 * 4 + 255
    for m in (12016, 1 << 20):
        assert size(m, 5120, 17408) <= 256 << 20 and size(m, 8192, 131072) <= 256 << 20
        assert size(m, 5120, 17408) >= size(m - 1, 5120, 17408) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,group", ((1025, 264, 128), (2500, 520, 32)))
def test_many_tokens_of_a_long_narrow_weight(M, N, group):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    K = 12416
    y, (x, cp, sp, b) = run(lib, M, N, K, group, True, 40)
    for m in (0, 1000, 1020, 1024, (M - 1) // 16 * 16):
        say(f"rows {m} .. of {M}")
        assert torch.equal(y[m:m + 16], lib.w8a8_w4_linear(x[m:m + 16].cuda(), cp, sp, N, group, b.cuda()))
