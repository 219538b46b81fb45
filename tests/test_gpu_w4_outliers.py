"""4-bit projections of tokens with elements far above the others, which the sums carry 136 to 144 times whatever their
codes are."""
import numpy as np
import pytest
import torch

import plain_decode as P
from parity import say
from test_gpu_w4 import weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


@pytest.mark.parametrize("group", (32, 64, 128))
@pytest.mark.parametrize("M,N,K", ((1, 48, 1280), (9, 264, 640), (40, 4096, 640), (256, 5120, 640)))
def test_whole_numbers_stay_exact_beside_large_ones(lib, M, N, K, group):
    """x = +-1 and one element of 2^14 in every group, scales of one: whole numbers below 2^24 throughout (144 * (2^14 + 127)
    = 2.4 million a group, 10 groups of 8 * 2^14 each in the total), so the only rounding is the output's."""
    say(f"w4 whole numbers M={M} N={N} K={K} group={group}")
    g = torch.Generator().manual_seed(M + group)
    x = torch.randint(0, 2, (M, K), generator=g) * 2 - 1
    x[:, torch.arange(0, K, group) + torch.randint(0, group, (K // group,), generator=g)] = 1 << 14
    codes, scales = weight(N, K, group, 2, full_range=True)
    cp, sp = lib.w8a8_w4_pack(codes.cuda(), torch.ones_like(scales).cuda())
    y = lib.w8a8_w4_linear(x.to(torch.bfloat16).cuda(), cp, sp, N, group)
    ref = torch.from_numpy(x.numpy() @ P.w4_codes(codes.numpy(), K).T)
    assert int(ref.abs().max()) < 1 << 24
    assert torch.equal(y.cpu(), ref.to(torch.float32).to(torch.bfloat16))


@pytest.mark.parametrize("by", (2.0 ** 7, 2.0 ** 14))
@pytest.mark.parametrize("M,group", ((1, 128), (16, 32), (40, 64)))
def test_large_elements(lib, M, group, by):
    """Every rounding of a group (at most one for each of its 2 * group products, of at most a unit of fp32) is of a sum
    below (136 + 144) * sum|x|."""
    N, K = 520, 1152
    say(f"w4 outliers M={M} group={group} by {by}")
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randperm(K, generator=g)[:12]] *= by
    x = x.to(torch.bfloat16)
    codes, scales = weight(N, K, group, 3)
    cp, sp = lib.w8a8_w4_pack(codes.cuda(), scales.cuda())
    y = lib.w8a8_w4_linear(x.cuda(), cp, sp, N, group).double().cpu().numpy()
    ref = P.w4_linear(x.float().numpy(), P.w4_codes(codes.numpy(), K), scales.float().numpy(), group, None)
    size = x.double().abs().numpy().reshape(M, K // group, group).sum(2)
    bound = 2 * group * 2.0 ** -23 * 280 * (size @ scales.double().numpy().T)
    err = np.abs(y - ref) - 2 ** -8 * np.abs(ref)
    say(f"largest error past bf16's: {(err / (size @ scales.double().numpy().T)).max() * 2 ** 17:.2f} * 2^-17 sum|x| scale")
    assert (err <= bound).all()
