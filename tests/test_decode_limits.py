"""Few-token calls past what a launch can hold are refused as shapes by the C entry points, and those below are not
(without a GPU a valid call ends at the device check; nothing is launched)."""
import pytest
import torch

from parity import say
from test_abi import A, DEVICE, SHAPE
from test_decode_abi import append, attend, lib as abi, read      # noqa: F401  (the C library, as a fixture)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a valid call would run")


@no_gpu
def test_limits_of_a_launch(abi):      # noqa: F811
    def w4(m, n):
        return abi.w8a8_w4_linear(A, A, A, None, A, m, n, 128, 64, None, 0, None)
    assert w4(1, (1 << 28) - 32) == DEVICE and w4(1, (1 << 28) - 24) == SHAPE and w4(1, 1 << 30) == SHAPE
    assert w4(1 << 20, 1 << 20) == DEVICE and w4(1 << 20, (1 << 20) + 8) == SHAPE
    wide = dict(ldk=1 << 20, ldv=1 << 20, width=1 << 16)
    assert append(abi, seqs=1, tokens=1 << 20, heads=127, page=16, **wide) == DEVICE
    assert append(abi, seqs=1, tokens=1 << 20, heads=128, page=16, **wide) == SHAPE
    assert append(abi, seqs=100, tokens=1 << 17, heads=8, page=16, **wide) == DEVICE       # several launches
    assert read(abi, seqs=1, length=(1 << 28) - 16, heads=1, dim=128) == DEVICE
    assert read(abi, seqs=1, length=1 << 28, heads=1, dim=128) == SHAPE
    assert attend(abi, seqs=1 << 14, tokens=1, q_heads=1024, heads=1024, ldq=1 << 16) == DEVICE    # several launches


@pytest.mark.gpu
def test_more_weights_than_one_launch_takes():
    """Quantizing and packing 2^35 weights and more: the first rows, those about the mark and the last are as by themselves."""
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    K, N, group = 131072, (1 << 18) + 40, 128
    say(f"w4 quantize and pack of {N} x {K}")
    at = [0, 1 << 17, (1 << 18) - 2048, (1 << 18) - 16, 1 << 18, (1 << 18) + 24]
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    for r in at:
        w[r:r + 16] = torch.randn(16, K, generator=g, device="cuda", dtype=torch.bfloat16)
    codes, scales = lib.w8a8_w4_quantize(w, group)
    alone = [lib.w8a8_w4_quantize(w[r:r + 16], group) for r in at]
    del w
    for r, (c, s) in zip(at, alone):
        assert torch.equal(codes[r:r + 16], c) and torch.equal(scales[r:r + 16], s) and c.any(), r
    cp, sp = lib.w8a8_w4_pack(codes, scales)
    del codes, scales
    cp, sp = cp.view(-1, 8 * K), sp.view(-1, 16 * K // group)
    for r, (c, s) in zip(at, alone):
        if r % 16 == 0:
            p, t = lib.w8a8_w4_pack(c, s)
            assert torch.equal(cp[r // 16], p) and torch.equal(sp[r // 16], t), r
    assert (cp[-1].view(K // 128, 4, 16, 16)[:, :, 8:] == 0x88).all()        # N % 16 == 8: the padding rows
    del cp, sp
    torch.cuda.empty_cache()
