"""E4M3 projections with block scales: quantizers bit for bit, products against 64 bits.

Tolerance of a product: what the matrix instruction may drop (each product of a block what lies 2^-13 below the block's largest:
measured on the device with products that cancel), fp32 additions of up to 16 groups within a block and of the blocks
(2^-20 + blocks * 2^-24 of the sum of magnitudes, with the scales' product), and half a step of bf16."""
import numpy as np
import pytest
import torch

import plain_layer as plain
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def inputs(M, N, K, seed, bias=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-3, 4, (M, 1)))
    x[:, rng.random(K) < 0.01] *= 20
    w = rng.standard_normal((N, K)) * 0.02 * np.exp2(rng.integers(-2, 3, (N, 1)))
    return plain.bf16(x), plain.bf16(w), plain.bf16(0.1 * rng.standard_normal(N)) if bias else None


def act_codes(x):
    v = x.float().numpy().reshape(-1, 128)
    s = np.abs(v).max(1) / np.float32(448)
    return plain.e4m3_codes(v, s).reshape(x.shape), s.reshape(x.shape[0], -1)


def weight_codes(w):
    N, K = w.shape
    v = w.float().numpy()
    q, s = np.zeros((N, K), np.uint8), np.zeros((-(-N // 128), K // 128), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            b = v[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            s[i, j] = np.abs(b).max() / np.float32(448)
            q[128 * i:128 * i + 128, 128 * j:128 * j + 128] = plain.e4m3_codes(b.reshape(1, -1), s[i:i + 1, j]).reshape(b.shape)
    return q, s


def check(y, q, s, w, sw, bias, what="", rows=None, cols=None):
    """Against 64 bits; `rows` and `cols`: these of y only."""
    if rows is not None:
        y, q, s = y[rows], q[rows], s[rows]
    if cols is not None:
        assert (np.diff(cols) > 0).all()
        block = cols // 128
        want, dropped, spread = (np.zeros((q.shape[0], len(cols))) for _ in range(3))
        for b in np.unique(block):
            at = block == b
            want[:, at], dropped[:, at], spread[:, at] = plain.block_product(q, s, w[cols[at]], sw[b:b + 1], None if bias is None else bias[cols[at]])
        y = y[:, cols]
    else:
        want, dropped, spread = plain.block_product(q, s, w, sw, bias)
    blocks = q.shape[1] // 128
    off = np.abs(plain.f64(y) - want)
    by = dropped + spread * (2.0 ** -20 + (blocks + 3) * 2.0 ** -24) + (np.abs(want) + dropped) * 2.0 ** -8 + 2.0 ** -134
    assert np.isfinite(plain.f64(y)).all() and (off <= by).all(), f"{what}: off by {np.max(off / by)} of what it may be"


def near(y, x, w, bias):
    """Every output, loosely: against fp32 products of the values."""
    (q, s), (wq, sw) = x, w
    (M, K), N = q.shape, wq.shape[0]
    v = (q.view(torch.float8_e4m3fn).float().view(M, -1, 128) * s[:, :, None]).view(M, K)
    ref = v @ (wq.view(torch.float8_e4m3fn).float().view(N, -1, 128) * sw.repeat_interleave(128, 0)[:N, :, None]).view(N, K).t()
    if bias is not None:
        ref = ref + bias.float()
    rms = ref.square().mean(1, keepdim=True).sqrt()          # a token's own: tokens differ by powers of two
    assert ((y.float() - ref).abs() <= ref.abs() * 2.0 ** -7 + rms * 2.0 ** -7).all()


def some(n, seed):
    """Some of n places: both ends, around every border of a tile, others."""
    rng = np.random.default_rng(seed)
    at = {0, n - 1, n // 2} | {b + d for b in (16, 32, 64, 128, 256, n // 64 * 64, n // 128 * 128, n // 256 * 256) for d in (-1, 0)} | set(rng.integers(0, n, 12).tolist())
    return np.array(sorted(i for i in at if 0 <= i < n))


@pytest.mark.parametrize("M,K", ((1, 128), (3, 256), (37, 1024), (300, 640), (2, 131072)))
def test_quantize_activations(lib, M, K):
    x, _, _ = inputs(M, 8, K, M + K)
    if M > 2:
        x[1, :128], x[2, 128:256] = 0, (x[2, 128:256].float() * 2.0 ** -100).to(torch.bfloat16)
    q, s = act_codes(x)
    gq, gs = lib.w8a8_quantize_act_block(x.cuda())
    assert np.array_equal(gq.cpu().numpy(), q) and np.array_equal(gs.cpu().numpy(), s)
    fill = torch.full((lib.packed_bytes(M, K),), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((K // 128, lib.block_scale_stride(M)), -1.0, device="cuda")
    lib.w8a8_quantize_act_block_packed(x.cuda(), out=(fill, scales))
    rows = plain.unpack(fill.cpu().numpy(), -(-M // 32) * 32, K)
    assert np.array_equal(rows[:M], q) and (rows[M:] == 0xAB).all()
    assert np.array_equal(scales.cpu().numpy()[:, :M].T, s) and (scales[:, M:] == -1).all()


@pytest.mark.parametrize("N,K", ((8, 128), (128, 256), (136, 384), (1000, 1024)))
def test_quantize_weights(lib, N, K):
    _, w, _ = inputs(1, N, K, N + K)
    w[:128, 128:256] = 0
    q, s = weight_codes(w)
    gq, gs = lib.w8a8_quantize_weight_block(w.cuda())
    assert np.array_equal(gs.cpu().numpy(), s) and np.array_equal(gq.cpu().numpy(), q)
    assert np.array_equal(lib.w8a8_pack_weight(gq).cpu().numpy(), plain.pack(q))


# every form: few tokens (16 and 32 weight rows a workgroup; 1, 2 and 4 blocks of tokens; fused), tiles of each size, parts of K, workgroups
# that walk over tiles; ragged last tiles, and blocks of columns fewer than the stages
SHAPES = ((7, 4360, 2048), (16, 8, 4096), (20, 4360, 256), (40, 4360, 384), (64, 40, 8192), (70, 8, 128), (66, 72, 4096), (100, 264, 5120), (130, 1032, 17408),
          (17, 8200, 6272), (70, 34824, 128), (129, 34824, 384), (300, 1032, 4096), (258, 5128, 2048), (520, 4104, 640), (1030, 8200, 256), (1, 8, 128), (1, 64, 256), (2, 136, 1024), (5, 24, 2176), (16, 256, 512), (17, 200, 384), (31, 128, 640), (33, 392, 256),
          (48, 264, 128), (64, 128, 1024), (65, 136, 512), (100, 520, 256), (129, 256, 384), (200, 72, 256), (257, 264, 128), (300, 136, 256),
          (1030, 8200, 128), (1700, 7160, 1152), (1000, 5128, 128), (740, 7160, 512), (834, 4104, 128), (834, 4104, 1024), (65, 17416, 256), (2300, 16392, 1152), (5000, 8200, 640))


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("bias", (False, True))
def test_linear(lib, M, N, K, bias):
    say(f"block linear {M} x {K} x {N}, bias {bias}")
    x, w, b = inputs(M, N, K, M + N + K, bias)
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    wp = lib.w8a8_pack_weight(wq)
    bc = None if b is None else b.cuda()
    y = lib.w8a8_fp8_block_linear_packed(x.cuda(), wp, N, sw, bc)
    q, s = act_codes(x)
    if M * N * K <= 1 << 25:
        check(y, q, s, wq.cpu().numpy(), sw.cpu().numpy(), b, "linear")
    else:
        check(y, q, s, wq.cpu().numpy(), sw.cpu().numpy(), b, "linear", some(M, N), some(N, M))
    near(y, lib.w8a8_quantize_act_block(x.cuda()), (wq, sw), bc)
    qp, sp = lib.w8a8_quantize_act_block_packed(x.cuda())
    assert torch.equal(lib.w8a8_fp8_block_gemm_packed(qp, sp, wp, sw, M, N, K, bc), y)


@pytest.mark.parametrize("M,N,K", ((1, 5120, 17408), (5, 5120, 17408), (64, 2056, 5120), (64, 5120, 17408), (100, 5120, 17408), (1502, 4096, 4096), (2270, 1160, 5120),
                                   (700, 17408, 1024), (4370, 4360, 640), (300, 65544, 512), (513, 33000, 1152), (189, 7176, 17408),
                                   (65, 7176, 17408), (17, 17416, 5120), (2270, 5120, 5120), (200, 4104, 17408), (17, 7176, 17408), (64, 34824, 5120), (65, 5120, 17408)))
def test_large(lib, M, N, K):
    """Sampled rows and columns of larger products."""
    say(f"block linear {M} x {K} x {N}")
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    wq, sw = lib.w8a8_quantize_weight_block((torch.randn(N, K, generator=g, device="cuda") * 0.02).to(torch.bfloat16))
    y = lib.w8a8_fp8_block_linear_packed(x, lib.w8a8_pack_weight(wq), N, sw)
    q, s = lib.w8a8_quantize_act_block(x)
    check(y, q.cpu().numpy(), s.cpu().numpy(), wq.cpu().numpy(), sw.cpu().numpy(), None, "large", some(M, N)[::3], some(N, M)[::2])
    near(y, (q, s), (wq, sw), None)


@pytest.mark.parametrize("M", (3, 40, 200))
def test_scales_far_apart_and_zero_blocks(lib, M):
    """Blocks 2^40 apart, and blocks of zeros: the sum over blocks is fp32."""
    x, w, b = inputs(M, 136, 768, 77)
    by = torch.tensor([1.0, 2.0 ** 20, 2.0 ** -20, 1.0, 0.0, 2.0 ** -60]).repeat_interleave(128)
    x, w = (x.float() * by).to(torch.bfloat16), (w.float() / torch.where(by > 0, by, 1.0) ** 1.5).to(torch.bfloat16)
    w[128:, 256:384] = 0
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    y = lib.w8a8_fp8_block_linear_packed(x.cuda(), lib.w8a8_pack_weight(wq), 136, sw, b.cuda())
    q, s = act_codes(x)
    check(y, q, s, wq.cpu().numpy(), sw.cpu().numpy(), b)
    zero = torch.zeros_like(x).cuda()
    assert torch.equal(lib.w8a8_fp8_block_linear_packed(zero, lib.w8a8_pack_weight(wq), 136, sw, b.cuda()), b.cuda().expand(M, 136))


@pytest.mark.parametrize("M", (1, 5, 16, 40, 64, 130, 300))
def test_tokens_that_are_not_finite_and_padding(lib, M):
    """A NaN or an infinity spoils its own token; what the padding of the packed codes and scales holds is not used."""
    N, K = 264, 512
    x, w, b = inputs(M, N, K, 5)
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    wp = lib.w8a8_pack_weight(wq)
    q, s = torch.full((lib.packed_bytes(M, K),), 0x7F, dtype=torch.uint8, device="cuda"), torch.full((K // 128, lib.block_scale_stride(M)), float("nan"), device="cuda")
    lib.w8a8_quantize_act_block_packed(x.cuda(), out=(q, s))
    y = lib.w8a8_fp8_block_gemm_packed(q, s, wp, sw, M, N, K, b.cuda())
    assert torch.equal(y, lib.w8a8_fp8_block_linear_packed(x.cuda(), wp, N, sw, b.cuda())) and torch.isfinite(y.float()).all()
    if M > 4:
        x[1, 7], x[3, 300] = float("nan"), float("inf")
        z = lib.w8a8_fp8_block_linear_packed(x.cuda(), wp, N, sw, b.cuda())
        keep = torch.tensor([i for i in range(M) if i not in (1, 3)], device="cuda")
        assert torch.equal(z[keep], y[keep])


def test_empty_and_refused(lib):
    x, w, b = inputs(4, 136, 256, 6)
    x, w, b = x.cuda(), w.cuda(), b.cuda()
    wq, sw = lib.w8a8_quantize_weight_block(w)
    wp = lib.w8a8_pack_weight(wq)
    f = lib.w8a8_fp8_block_linear_packed
    assert f(x[:0], wp, 136, sw, b).shape == (0, 136)
    with pytest.raises(ValueError, match="s_w"):
        f(x, wp, 136, sw[:1].contiguous())
    with pytest.raises(ValueError, match="packed weight"):
        f(x, wp[:-1].contiguous(), 136, sw)
    with pytest.raises(ValueError, match="bias"):
        f(x, wp, 136, sw, b[:8].contiguous())
    with pytest.raises(lib.W8A8Error, match="BAD_SHAPE"):
        f(x, wp, 132, sw)
    with pytest.raises(ValueError, match="workspace"):
        f(x, wp, 136, sw, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        f(x, wp.view(torch.int8), 136, sw)
    with pytest.raises(ValueError, match="inconsistent"):
        q, s = lib.w8a8_quantize_act_block_packed(x)
        lib.w8a8_fp8_block_gemm_packed(q, s[:, :4].contiguous(), wp, sw, 4, 136, 256)
    with pytest.raises(lib.W8A8Error, match="BAD_SHAPE"):
        lib.w8a8_quantize_act_block(x[:, :64].contiguous())


@pytest.mark.parametrize("M", (1, 20, 150))
def test_captured_on_another_stream_and_outputs_given(lib, M):
    N, K = 392, 640
    x, w, b = inputs(M, N, K, 8)
    x, b = x.cuda(), b.cuda()
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    wp = lib.w8a8_pack_weight(wq)
    want = lib.w8a8_fp8_block_linear_packed(x, wp, N, sw, b)
    ws = torch.empty(lib.fp8_block_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        assert torch.equal(lib.w8a8_fp8_block_linear_packed(x, wp, N, sw, b, workspace=ws, out=out), want)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        lib.w8a8_fp8_block_linear_packed(x, wp, N, sw, b, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        ws.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
