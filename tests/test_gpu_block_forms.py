"""Block products whose K is cut into parts, two calls at once."""
import pytest
import torch

from parity import say
from test_gpu_fp8_block import inputs, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


@pytest.mark.parametrize("M,N,K", ((130, 1032, 17408), (100, 5128, 17408), (66, 72, 4096)))
def test_two_streams_at_once(lib, M, N, K):
    """Calls that overlap, each with partial sums in a workspace of its own."""
    say(f"block linear {M} x {K} x {N} on two streams")
    parts = lib.fp8_block_gemm_workspace_bytes(M, N, K) // (4 * M * N)
    assert parts > 1
    x, w, b = inputs(M, N, K, 31)
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    wp, b = lib.w8a8_pack_weight(wq), b.cuda()
    xs = [x.cuda(), (x.flip(0) * 2).cuda()]
    want = [lib.w8a8_fp8_block_linear_packed(v, wp, N, sw, b) for v in xs]
    near(want[0], lib.w8a8_quantize_act_block(xs[0]), (wq, sw), b)
    codes = [lib.w8a8_quantize_act_block_packed(v) for v in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [[], []]
        for _ in range(8):
            for s, c, g in zip(streams, codes, got):
                with torch.cuda.stream(s):
                    g.append(lib.w8a8_fp8_block_gemm_packed(*c, wp, sw, M, N, K, b))
        torch.cuda.synchronize()
        assert all(torch.equal(y, t) for ys, t in zip(got, want) for y in ys)
