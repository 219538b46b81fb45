"""The 4-bit-weight projection on the GPU against its formula in 64 bits.

Tolerance.  The output is rounded once to bf16 (half a unit: 2^-9 of the value).  The sums are fp32: within
a group the running sum is that of x times (136 + code), started at -136 sum(x), so a rounding is 2^-24 of up
to ~1,500 sigma where the whole row's result is ~2.6 sqrt(K) sigma; about a hundred of them, random, leave
below 1e-4 of the outputs' rms.  So |y - ref| <= 2^-8 |ref| + 1e-3 rms(ref) holds every element."""
import numpy as np
import pytest
import torch

import plain_decode as P
import workloads as W
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def weight(N, K, group, seed, full_range=False):
    """Row-major codes (uint8 [N, K / 2]) and scales (bf16 [N, K / group]) on the CPU."""
    g = torch.Generator().manual_seed(seed)
    if full_range:
        c = torch.randint(0, 16, (N, K), generator=g, dtype=torch.int64)
    else:
        c = (torch.randn(N, K, generator=g) * 2.6).round().clamp(-7, 7).to(torch.int64) + 8
    codes = (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8).contiguous()
    scales = (0.005 + 0.01 * torch.rand(N, K // group, generator=g)).to(torch.bfloat16)
    return codes, scales


def check(y, ref, what):
    y = y.float().cpu().numpy().astype(np.float64)
    rms = np.sqrt(np.mean(ref ** 2))
    over = np.abs(y - ref) - (2 ** -8 * np.abs(ref) + 1e-3 * rms)
    assert np.isfinite(y).all() and over.max() <= 0, f"{what}: {(over > 0).sum()} of {over.size} off, by up to {over.max()}"


def run(lib, M, N, K, group, bias, seed, full_range=False, x=None):
    say(f"w4 M={M} N={N} K={K} group={group} bias={bias}")
    codes, scales = weight(N, K, group, seed, full_range)
    if x is None:
        x = W.make_inputs(W.custom("linear", M, K, 8, seed=seed)).x
    b = (torch.randn(N, generator=torch.Generator().manual_seed(seed + 1))).to(torch.bfloat16) if bias else None
    cp, sp = lib.w8a8_w4_pack(codes.cuda(), scales.cuda())
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = lib.w8a8_w4_linear(x.cuda(), cp, sp, N, group, None if b is None else b.cuda(), out=out)
    torch.cuda.synchronize()
    ref = P.w4_linear(x.float().numpy(), P.w4_codes(codes.numpy(), K), scales.float().numpy(), group,
                      None if b is None else b.float().numpy())
    check(y, ref, "w4")
    return y, (x, cp, sp, b)


@pytest.mark.parametrize("group", (32, 64, 128))
@pytest.mark.parametrize("M", (1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 130))
def test_tokens(lib, M, group):
    run(lib, M, 104, 640, group, M % 2 == 0, seed=M)


@pytest.mark.parametrize("N", (8, 16, 24, 40, 264, 1000))
@pytest.mark.parametrize("K", (128, 256, 1024, 1152, 2176))
def test_shapes(lib, N, K):
    run(lib, 3, N, K, 32 if K % 256 else 128, True, seed=N + K, full_range=True)


@pytest.mark.parametrize("M,N,K,group", ((1, 1024, 1024, 128), (5, 5120, 17408, 32), (64, 5120, 5120, 64), (1, 17408, 5120, 128), (16, 12288, 512, 32), (40, 264, 12544, 128)))
def test_projection_sizes(lib, M, N, K, group):
    run(lib, M, N, K, group, True, seed=7)


@pytest.mark.parametrize("N,K,group", ((40, 256, 32), (1024, 1024, 128), (520, 2176, 64), (104, 16384, 32), (8264, 640, 128)))
def test_a_token_alone_and_in_a_batch(lib, N, K, group):
    """Bit for bit the same, whichever form of the kernel the batch runs."""
    y, (x, cp, sp, b) = run(lib, 70, N, K, group, True, seed=3)
    for rows in (slice(0, 1), slice(5, 21), slice(30, 62), slice(6, 70)):
        part = lib.w8a8_w4_linear(x[rows].contiguous().cuda(), cp, sp, N, group, b.cuda())
        assert torch.equal(part.view(torch.int16), y[rows].view(torch.int16)), rows


# 1 to 4 row blocks a workgroup: few rows, rows in one round of the CUs, in several, in splits
@pytest.mark.parametrize("M,N,K,group", ((5, 4096, 640, 64), (16, 5120, 1152, 128), (9, 12288, 384, 32), (16, 12280, 1152, 64), (7, 16384, 256, 128), (16, 34816, 128, 32), (13, 5120, 12416, 64), (16, 16400, 640, 128)))
def test_up_to_sixteen_tokens(lib, M, N, K, group):
    y, (x, cp, sp, b) = run(lib, M, N, K, group, True, 700 + M)
    for m in (0, M - 1):
        one = lib.w8a8_w4_linear(x[m:m + 1].cuda(), cp, sp, N, group, b.cuda())
        assert torch.equal(y[m:m + 1], one), f"row {m} of {M} differs from the row alone"


# 17 tokens and more: 2, 3 and 4 row blocks an item, items that a workgroup takes one after another, runs without a
# block (K < 1024), K in splits; and the tile of x shared by 4 .. 7 and by 8 .. 12 waves
@pytest.mark.parametrize("M,N,K,group", ((64, 4096, 640, 64), (64, 5120, 1152, 128), (24, 34816, 256, 32), (256, 4096, 1152, 128), (250, 4088, 384, 32), (20, 5128, 12416, 64), (129, 2056, 12288, 32), (256, 5120, 640, 64), (500, 4096, 384, 32), (490, 4104, 1280, 128)))
def test_many_tokens(lib, M, N, K, group):
    y, (x, cp, sp, b) = run(lib, M, N, K, group, True, 900 + M)
    few = [lib.w8a8_w4_linear(x[m:m + 16].cuda(), cp, sp, N, group, b.cuda()) for m in (0, 16, (M - 1) // 16 * 16)]
    for m, f in zip((0, 16, (M - 1) // 16 * 16), few):
        assert torch.equal(y[m:m + 16], f), f"rows {m} .. of {M} differ from the same rows alone"


def test_whole_numbers_are_exact(lib):
    """x = +-1 and scales of one: sums of whole numbers below 2^24, so the only rounding is the output's."""
    K, N = 1280, 48
    x = torch.randint(0, 2, (9, K), generator=torch.Generator().manual_seed(1)) * 2 - 1
    codes, scales = weight(N, K, 64, 2, full_range=True)
    cp, sp = lib.w8a8_w4_pack(codes.cuda(), torch.ones_like(scales).cuda())
    y = lib.w8a8_w4_linear(x.to(torch.bfloat16).cuda(), cp, sp, N, 64)
    ref = torch.from_numpy(x.numpy() @ P.w4_codes(codes.numpy(), K).T).to(torch.bfloat16)
    assert torch.equal(y.cpu(), ref)


def test_large_and_tiny_values(lib):
    for by in (2.0 ** 60, 2.0 ** -60):
        x = (torch.randn(4, 512, generator=torch.Generator().manual_seed(2)) * by).to(torch.bfloat16)
        run(lib, 4, 64, 512, 128, False, seed=11, x=x)


@pytest.mark.parametrize("N,K,group", ((24, 256, 32), (16, 128, 64), (264, 640, 128)))
def test_pack_layout(lib, N, K, group):
    codes, scales = weight(N, K, group, 5, full_range=True)
    cp, sp = (t.cpu() for t in lib.w8a8_w4_pack(codes.cuda(), scales.cuda()))
    rows = -(-N // 16) * 16
    assert cp.numel() == lib.w4_code_bytes(N, K) == rows * K // 2
    assert 2 * sp.numel() == lib.w4_scale_bytes(N, K, group) == rows * (K // group) * 2
    c, packed = P.w4_codes(codes.numpy(), K), cp.numpy()
    for n in range(rows):
        for k in range(0, K, 3):
            byte, shift = P.w4_packed_byte(n, k, K)
            assert (int(packed[byte]) >> shift & 15) - 8 == (c[n, k] if n < N else 0), (n, k)
    s = sp.view(rows // 16, K // group, 16).permute(0, 2, 1).reshape(rows, -1)
    assert torch.equal(s[:N], scales) and not s[N:].any()


@pytest.mark.parametrize("group", (32, 64, 128))
def test_quantize(lib, group):
    """Scales bf16(amax / 7), codes RNE(w / scale) to +-7: bit for bit against single fp32 operations."""
    N, K = 37, 768
    w = (torch.randn(N, K, generator=torch.Generator().manual_seed(group)) * 0.02).to(torch.bfloat16)
    w[3] = 0
    w[5, :group] *= 2.0 ** -100
    w[7] = 1e-40                                            # scales that are bf16 subnormals, or zero
    codes, scales = lib.w8a8_w4_quantize(w.cuda(), group)
    g = w.float().numpy().reshape(N, K // group, group)
    s = torch.from_numpy(np.abs(g).max(2) / np.float32(7)).to(torch.bfloat16)
    assert torch.equal(scales.cpu().view(torch.int16), s.view(torch.int16))
    sf = s.float().numpy()[:, :, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(sf > 0, np.clip(np.rint(g / sf), -7, 7), 0).reshape(N, K)
    assert np.array_equal(P.w4_codes(codes.cpu().numpy(), K), c.astype(np.int64))


def test_quantized_weight_end_to_end(lib):
    """Quantize, pack, multiply: within the weight's rounding (half a step each, random signs) of x W^T."""
    N, K, M = 256, 2048, 5
    w = (torch.randn(N, K, generator=torch.Generator().manual_seed(1)) * 0.02).to(torch.bfloat16)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    codes, scales = lib.w8a8_w4_quantize(w.cuda(), 32)
    y = lib.w8a8_w4_linear(x.cuda(), *lib.w8a8_w4_pack(codes, scales), N, 32).double().cpu()
    ref = x.double() @ w.double().t()
    step = scales.double().cpu().mean()
    assert float((y - ref).norm()) <= 1.5 * float(step) / 12 ** 0.5 * K ** 0.5 * (M * N) ** 0.5


@pytest.mark.parametrize("M,N,K", ((3, 264, 640), (16, 4096, 384), (40, 1000, 1152), (256, 5120, 640)))
def test_a_token_that_is_not_finite_spoils_its_own_row_only(lib, M, N, K):
    y, (x, cp, sp, b) = run(lib, M, N, K, 64, True, 31)
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[M // 2, K // 3] = bad
        out = lib.w8a8_w4_linear(z.cuda(), cp, sp, N, 64, b.cuda())
        others = torch.arange(M, device="cuda") != M // 2
        assert torch.equal(out[others], y[others]) and not torch.isfinite(out[M // 2].float()).any()


def test_offsets_past_2_31_bytes(lib):
    """A packed weight of 2.2 GB: the rows on both sides of the 2^31-byte mark and the last ones."""
    K, N, group = 131072, 33600, 128
    say("w4 codes past 2^31 bytes")
    g = torch.Generator(device="cuda").manual_seed(1)
    cp = torch.randint(0, 256, (lib.w4_code_bytes(N, K),), generator=g, dtype=torch.uint8, device="cuda")
    sp = (torch.rand(lib.w4_scale_bytes(N, K, group) // 2, generator=g, device="cuda") * 0.01).to(torch.bfloat16)
    x = torch.randn(2, K, generator=g, device="cuda").to(torch.bfloat16)
    y = lib.w8a8_w4_linear(x, cp, sp, N, group).float().cpu().numpy()
    block = 2 ** 31 // (K // 128 * 1024)                    # the block of 16 rows that starts at the mark
    assert 16 * block < N
    for b in (0, block - 1, block, N // 16 - 1):
        words = cp.view(-1, K // 128, 4, 16, 4, 4)[b].cpu().numpy()
        codes = np.empty((16, K), dtype=np.int64)
        cols = np.arange(K)
        for r in range(16):
            j = cols % 8
            byte = words[cols // 128, cols // 8 % 4, r, cols // 32 % 4, 2 * (j % 2) + j // 4]
            codes[r] = (byte >> (4 * (j // 2 % 2)) & 15).astype(np.int64) - 8
        s = sp.view(-1, K // group, 16)[b].float().cpu().numpy().T
        ref = P.w4_linear(x.float().cpu().numpy(), codes, s, group, None)
        check(torch.from_numpy(y[:, 16 * b:16 * b + 16]), ref, f"block {b}")


def test_refusals(lib):
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    codes, scales = weight(16, 256, 64, 1)
    cp, sp = lib.w8a8_w4_pack(codes.cuda(), scales.cuda())
    ok = lib.w8a8_w4_linear(x, cp, sp, 16, 64)
    assert ok.shape == (2, 16)
    assert lib.w8a8_w4_linear(x[:0], cp, sp, 16, 64).shape == (0, 16)
    with pytest.raises(TypeError):
        lib.w8a8_w4_linear(x.float(), cp, sp, 16, 64)
    with pytest.raises(TypeError):
        lib.w8a8_w4_linear(x, cp.view(torch.int8), sp, 16, 64)
    with pytest.raises(ValueError):
        lib.w8a8_w4_linear(x.t(), cp, sp, 16, 64)
    with pytest.raises(ValueError):
        lib.w8a8_w4_linear(x, cp, sp, 24, 64)               # the packed weight has 16 rows
    with pytest.raises(ValueError):
        lib.w8a8_w4_linear(x, cp, sp, 16, 32)               # too few scales
    with pytest.raises(ValueError):
        lib.w8a8_w4_linear(x, cp, sp, 16, 48)
    with pytest.raises(ValueError):
        lib.w8a8_w4_linear(x, cp, sp, 16, 64, bias=torch.zeros(8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.W8A8Error):
        lib.w8a8_w4_linear(x, cp, sp, 12, 64)               # N % 8
    with pytest.raises(lib.W8A8Error):
        lib.w8a8_w4_linear(x.reshape(-1)[4:132].view(1, 128), cp, sp, 16, 128)     # misaligned
    with pytest.raises(ValueError):
        lib.w8a8_w4_linear(x, cp.cpu(), sp, 16, 64)
    with pytest.raises(ValueError):
        lib.w8a8_w4_quantize(x, 16)
    with pytest.raises(lib.W8A8Error):
        lib.w8a8_w4_quantize(torch.zeros(2, 192, dtype=torch.bfloat16, device="cuda"), 64)
    with pytest.raises(ValueError):
        lib.w8a8_w4_pack(codes.cuda(), scales[:8].contiguous().cuda())
