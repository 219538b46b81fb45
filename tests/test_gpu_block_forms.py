"""Block products in every tile, whole and with K in parts, and calls of the latter at once."""
import pytest
import torch

from block_forms import FORMS
from parity import say
from test_gpu_fp8_block import check, inputs, near, some

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


@pytest.mark.parametrize("M,N,K,tile,parts", FORMS)
def test_forms(lib, M, N, K, tile, parts):
    say(f"block linear {M} x {K} x {N}: {tile[0]} x {tile[1]} in {parts}")
    assert lib.fp8_block_gemm_workspace_bytes(M, N, K) // (4 * M * N) == (parts if parts > 1 else 0)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16)
    wq, sw = lib.w8a8_quantize_weight_block((torch.randn(N, K, generator=g, device="cuda") * 0.02).to(torch.bfloat16))
    y = lib.w8a8_fp8_block_linear_packed(x, lib.w8a8_pack_weight(wq), N, sw, b)
    q, s = lib.w8a8_quantize_act_block(x)
    check(y, q.cpu().numpy(), s.cpu().numpy(), wq.cpu().numpy(), sw.cpu().numpy(), b, "forms", some(M, N)[::3], some(N, M)[::2])
    near(y, (q, s), (wq, sw), b)


@pytest.mark.parametrize("M,N,K", ((5, 64, 131072), (20, 136, 131072), (139, 136, 131072), (16, 1032, 4096), (16, 1032, 4224)))
def test_long_rows(lib, M, N, K):
    """The longest rows, and rows on both sides of where tokens are quantized in every workgroup."""
    say(f"block linear {M} x {K} x {N}")
    x, w, b = inputs(M, N, K, 41)
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    wp = lib.w8a8_pack_weight(wq)
    y = lib.w8a8_fp8_block_linear_packed(x.cuda(), wp, N, sw, b.cuda())
    q, s = lib.w8a8_quantize_act_block(x.cuda())
    check(y, q.cpu().numpy(), s.cpu().numpy(), wq.cpu().numpy(), sw.cpu().numpy(), b, "long rows", some(M, N)[::4], some(N, M)[::4])
    near(y, (q, s), (wq, sw), b.cuda())
    qp, sp = lib.w8a8_quantize_act_block_packed(x.cuda())
    assert torch.equal(lib.w8a8_fp8_block_gemm_packed(qp, sp, wp, sw, M, N, K, b.cuda()), y)
