"""Norms, rotary positions and block-scaled projections where elements, bytes or tiles pass 32 bits, on two streams at once, and with
workspaces of their own in two graphs."""
import numpy as np
import pytest
import torch

import plain_layer as plain
from parity import say
from test_gpu_fp8_block import check, inputs, near
from test_gpu_norm import R_TOL, cuda
from test_gpu_norm import inputs as norm_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def filled(rows, width, seed):
    """bf16 [rows, width] of blocks of random rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    some = torch.randn(1024, width, generator=g, device="cuda").to(torch.bfloat16)
    for a in range(0, rows, 1024):
        x[a:a + 1024] = some[:min(1024, rows - a)]
        some = some.roll(1, 0)
    return x


def test_norm_past_32_bits(lib):
    """5.2 GB of x and of y; codes past 2^31 bytes."""
    M, K = 40003, 65536
    say(f"norm {M} x {K}")
    x, w = filled(M, K, 1), (1 + 0.1 * torch.randn(K, device="cuda")).to(torch.bfloat16)
    rows = torch.tensor([0, 16383, 16384, 32767, 32768, 32769, M - 2, M - 1], device="cuda")
    want, z, r, _ = plain.norm(x[rows].cpu(), None, w.cpu(), 1e-6)
    y = lib.w8a8_rmsnorm(x, w)[0]
    off = np.abs(plain.f64(y[rows]) - want)
    assert (off <= np.abs(want) * (2.0 ** -8 + R_TOL)).all()
    del y
    q, s, _ = lib.w8a8_rmsnorm_quantize_block_packed(x, w)
    v = z.astype(np.float32).reshape(-1, 128)
    sz = np.abs(v).max(1) / np.float32(448)
    at, k = rows.cpu()[:, None].long(), torch.arange(K)
    place = (at // 32 * (K // 64) + k // 64) * 2048 + at % 32 * 64 + k % 64
    got = q[place.cuda()].cpu().numpy()
    assert np.array_equal(got.reshape(-1, 128), plain.e4m3_codes(v, sz))
    scales = s[:, rows].t().cpu().numpy().astype(np.float64)
    expect = sz.astype(np.float64).reshape(scales.shape) * r
    assert (np.abs(scales - expect) <= expect * R_TOL).all()


def test_rope_past_32_bits(lib):
    seqs, tokens, heads, dim = 3, 80001, 64, 160
    say(f"rope {seqs} x {tokens}, {heads} heads of {dim}")
    x = filled(seqs * tokens, heads * dim, 2).view(seqs, tokens, heads, dim)
    assert x.numel() > 1 << 31
    lens, plan = [tokens + 7, tokens, 1000], lib.rope(128)
    y, none = lib.w8a8_rope(x, None, torch.tensor(lens, dtype=torch.int32).cuda(), plan)
    assert none is None
    for t in (0, tokens - 1000, tokens // 2, tokens - 1):
        want, spread = plain.turned(plain.f64(x[:, t:t + 1]), [n - tokens + t + 1 for n in lens], [int(v) for v in plan.turns.tolist()], False, 1.0)
        off = np.abs(plain.f64(y[:, t:t + 1]) - want)
        assert (off <= np.where(spread > 0, spread * 2.0 ** -21 + np.abs(want) * 2.0 ** -8 + 2.0 ** -134, 0.0)).all(), t


@pytest.mark.parametrize("M,N,K", ((70003, 34816, 128), (70001, 32768, 512), (70, 2200008, 256), (2100000, 1032, 512), (9, 2200008, 256)))
def test_products_past_32_bits(lib, M, N, K):
    """Outputs past 2^31 elements, weights of more rows than a tile's outputs may lie apart, more tokens than 2^21."""
    say(f"block product {M} x {K} x {N}")
    x, w = filled(M, K, M % 97), filled(N, K, N % 89)
    w *= 0.02
    b = torch.randn(N, device="cuda").to(torch.bfloat16)
    wq, sw = lib.w8a8_quantize_weight_block(w)
    del w
    y = lib.w8a8_fp8_block_linear_packed(x, lib.w8a8_pack_weight(wq), N, sw, b)
    rng = np.random.default_rng(3)
    rows = np.unique(np.concatenate(([0, M - 1, M // 2], rng.integers(0, M, 5))))
    cols = np.unique(np.concatenate(([0, N - 1, N // 2, N // 128 * 128 - 1], rng.integers(0, N, 40))))
    q, s = lib.w8a8_quantize_act_block(x[torch.from_numpy(rows).cuda()])
    got = y[torch.from_numpy(rows).cuda()].cpu()
    for c in cols:
        check(got[:, c:c + 1], q.cpu().numpy(), s.cpu().numpy(), wq[c:c + 1].cpu().numpy(), sw[c // 128:c // 128 + 1].cpu().numpy(), b[c:c + 1].cpu(), f"column {c}")


def test_two_streams_at_once(lib):
    """Calls that overlap: nothing is shared between them."""
    M, N, K = 200, 5120, 4096                                # (parts of K: partial sums in each call's own workspace)
    x, w, b = inputs(M, N, K, 31)
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    wp, b = lib.w8a8_pack_weight(wq), b.cuda()
    xs = [x.cuda(), (x.flip(0) * 2).cuda()]
    nx, res, nw = cuda(*norm_inputs(300, 4096, 32))
    want = [lib.w8a8_fp8_block_linear_packed(v, wp, N, sw, b) for v in xs]
    near(want[0], lib.w8a8_quantize_act_block(xs[0]), (wq, sw), b)
    norm = lib.w8a8_rmsnorm_quantize(nx, nw, res, rot_block=128)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, v in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append([lib.w8a8_fp8_block_linear_packed(v, wp, N, sw, b) for _ in range(4)])
        with torch.cuda.stream(streams[2]):
            n = lib.w8a8_rmsnorm_quantize(nx, nw, res, rot_block=128)
        torch.cuda.synchronize()
        assert all(torch.equal(y, t) for ys, t in zip(got, want) for y in ys)
        assert all(torch.equal(u, v) for u, v in zip(n, norm))


def test_two_graphs_that_share_a_workspace(lib):
    """Replayed one after the other on one stream, they may: each call writes what it reads."""
    N, K = 1032, 17408
    x, w, b = inputs(130, N, K, 33)
    wq, sw = lib.w8a8_quantize_weight_block(w.cuda())
    wp, b, x = lib.w8a8_pack_weight(wq), b.cuda(), x.cuda()
    ws = torch.empty(lib.fp8_block_workspace_bytes(130, N, K), dtype=torch.uint8, device="cuda")
    assert lib.fp8_block_gemm_workspace_bytes(130, N, K) > 0 and ws.numel() >= lib.fp8_block_workspace_bytes(40, N, K)
    outs = [torch.empty(m, N, dtype=torch.bfloat16, device="cuda") for m in (130, 40)]
    want = [lib.w8a8_fp8_block_linear_packed(x[:m], wp, N, sw, b) for m in (130, 40)]
    torch.cuda.synchronize()
    graphs, side = [], torch.cuda.Stream()
    for m, out in zip((130, 40), outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            lib.w8a8_fp8_block_linear_packed(x[:m], wp, N, sw, b, workspace=ws, out=out)
    for _ in range(4):
        for g, out in zip(graphs, outs):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, t) for o, t in zip(outs, want))
