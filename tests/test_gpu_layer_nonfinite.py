"""What the block quantizers, the products behind them and the norms leave of a value that is not finite: it shows in every
output that the formula makes of it, and nowhere else."""
import numpy as np
import pytest
import torch

from parity import say
from test_gpu_fp8_block import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


NAN, INF = float("nan"), float("inf")


# columns: a piece a thread, two of them, and 16 with threads behind the row's end
@pytest.mark.parametrize("M,K", ((5, 512), (300, 4096), (300, 8192), (5, 67584)))
@pytest.mark.parametrize("packed", (False, True))
def test_activations(lib, M, K, packed):
    """A block of 128 columns with a NaN has a NaN for its scale, wherever in the block it is and whatever its sign; all others stay."""
    say(f"block quantizer {M} x {K}, packed {packed}")
    x, _, _ = inputs(M, 8, K, K)
    spoiled = x.clone()
    spoiled[1, 7], spoiled[2, K - 1], spoiled[3, 128:256] = NAN, -NAN, NAN
    spoiled[4, 256 + 63], spoiled[4, 256 + 64] = INF, NAN
    f = lib.w8a8_quantize_act_block_packed if packed else lib.w8a8_quantize_act_block
    (q, s), (p, t) = f(x.cuda()), f(spoiled.cuda())
    if packed:
        q, p = lib.unpack_rows(q, M, K), lib.unpack_rows(p, M, K)
        s, t = s.t()[:M], t.t()[:M]
    at = torch.zeros(M, K // 128, dtype=torch.bool, device="cuda")
    at[1, 0] = at[2, -1] = at[3, 1] = at[4, 2] = True
    assert torch.equal(torch.isnan(t), at)
    assert torch.equal(t[~at], s[~at]) and torch.equal(p.view(M, -1, 128)[~at], q.view(M, -1, 128)[~at])


@pytest.mark.parametrize("N", (128, 136, 392))
def test_weights(lib, N):
    """A block of 128 x 128 with a NaN, and so for one that is nothing else."""
    K = 384
    _, w, _ = inputs(1, N, K, N)
    spoiled = w.clone()
    spoiled[N - 1, 130] = -NAN
    spoiled[:128, 256:] = NAN
    (q, s), (p, t) = lib.w8a8_quantize_weight_block(w.cuda()), lib.w8a8_quantize_weight_block(spoiled.cuda())
    at = torch.zeros_like(s, dtype=torch.bool)
    at[-1, 1] = at[0, 2] = True
    assert torch.equal(torch.isnan(t), at) and torch.equal(t[~at], s[~at])
    rows = at.repeat_interleave(128, 0)[:N]
    assert torch.equal(p.view(N, -1, 128)[~rows], q.view(N, -1, 128)[~rows])


# made in every workgroup and by a launch of its own, few tokens of 16 and 32 weight rows, tiles, parts of K
@pytest.mark.parametrize("M,N,K", ((5, 264, 512), (16, 1032, 1024), (5, 5128, 2176), (12, 2056, 8192), (20, 264, 512), (40, 4360, 384), (64, 264, 640), (130, 264, 512),
                                   (300, 1032, 4096), (700, 4104, 640), (2300, 16392, 640)))
def test_products(lib, M, N, K):
    """Every output of a token with a NaN is one, and none of a token with an infinity is finite; of a weight's block with a NaN, every
    output of its rows."""
    say(f"block linear {M} x {K} x {N}")
    x, w, b = inputs(M, N, K, 5)
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    wp, b = lib.w8a8_pack_weight(wq), b.cuda()
    y = lib.w8a8_fp8_block_linear_packed(x.cuda(), wp, N, sw, b)
    spoiled = x.clone()
    spoiled[1, 7], spoiled[2, K - 128:], spoiled[3, 300], spoiled[4, 64:66] = NAN, -NAN, -INF, torch.tensor([INF, NAN])
    z = lib.w8a8_fp8_block_linear_packed(spoiled.cuda(), wp, N, sw, b)
    assert torch.isnan(z[[1, 2, 4]].float()).all() and not torch.isfinite(z[3].float()).any()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[1:5] = False
    assert torch.equal(z[keep], y[keep])
    q, s = lib.w8a8_quantize_act_block_packed(spoiled.cuda())
    assert torch.equal(lib.w8a8_fp8_block_gemm_packed(q, s, wp, sw, M, N, K, b).view(torch.int16)[keep], y.view(torch.int16)[keep])
    w[N - 1, K - 1] = NAN
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    z = lib.w8a8_fp8_block_linear_packed(x.cuda(), lib.w8a8_pack_weight(wq), N, sw, b)
    first = (N - 1) // 128 * 128
    assert torch.isnan(z[:, first:].float()).all() and torch.equal(z[:, :first], y[:, :first])


def norm_inputs(M, K, seed):
    rng = np.random.default_rng(seed)
    x, r, w = rng.standard_normal((M, K)), rng.standard_normal((M, K)), 1 + 0.3 * rng.standard_normal(K)
    return [torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).cuda() for a in (x, r, w)]


# rows of one wave and of several, more than registers hold, threads behind the row's end
@pytest.mark.parametrize("M,K", ((1, 128), (5, 1152), (300, 5120), (3, 67584)))
@pytest.mark.parametrize("form,rot", (("int8", 0), ("int8", 128), ("fp8", 0), ("fp8", 128), ("block", 0)))
@pytest.mark.parametrize("packed", (False, True))
@pytest.mark.parametrize("value", (NAN, -NAN, INF))
def test_a_norms_weight(lib, M, K, form, rot, packed, value):
    """Codes behind a norm's weight with a value that is not finite: no scale over it is; scales of other blocks stay."""
    say(f"norm {M} x {K} {form}, rotated {rot}, packed {packed}, {value} in its weight")
    x, res, w = norm_inputs(M, K, K)
    name = {"int8": "w8a8_rmsnorm_quantize", "fp8": "w8a8_rmsnorm_quantize_fp8", "block": "w8a8_rmsnorm_quantize_block"}[form]
    f = getattr(lib, name + ("_packed" if packed else ""))
    more = {} if form == "block" else dict(rot_block=rot)
    _, s, h = f(x, w, res, **more)
    at = K - 70 if M > 1 else 3
    spoiled = w.clone()
    spoiled[at] = value
    _, t, g = f(x, spoiled, res, **more)
    if form == "block":
        s, t = (s.t()[:M], t.t()[:M]) if packed else (s, t)
        assert not torch.isfinite(t[:, at // 128]).any() and (value == INF or torch.isnan(t[:, at // 128]).all())
        keep = torch.arange(K // 128, device="cuda") != at // 128
        assert torch.equal(t[:, keep], s[:, keep])
    else:
        assert not torch.isfinite(t).any() and (value == INF or torch.isnan(t).all())
    assert torch.equal(g, h)
