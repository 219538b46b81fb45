"""The root-mean-square norm in all its outputs against 64 bits.

Tolerances.  z = h * weight is exact in fp32 and the codes depend on z alone, so codes without the rotation and their own
scales' numerators match bit for bit.  r: a lane adds up to 32 squares into each of four sums, then at most 4 + 16 + 6
partial sums meet: 58 roundings of 2^-24, halved by the root, and one each for the mean, eps, root and reciprocal: 33 * 2^-24 <
2^-18.  A product with r adds 2^-24: 2^-17.9 in all.  Rotated values are off by seven additions and a product of at most
2^-24 of the block's sum of magnitudes over sqrt(128) each: 2^-21 of it."""
import numpy as np
import pytest
import torch

import plain_layer as plain
from parity import say

pytestmark = pytest.mark.gpu

R_TOL = 2.0 ** -17
ROT_TOL = 2.0 ** -21


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def inputs(M, K, seed, residual=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-6, 6, (M, 1)))
    x[:, rng.random(K) < 0.02] *= 30
    r = rng.standard_normal((M, K)) * 2
    return plain.bf16(x), plain.bf16(r) if residual else None, plain.bf16(1 + 0.3 * rng.standard_normal(K))


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def close(got, want, by, what):
    off = np.abs(got - want)
    assert np.isfinite(got).all() and (off <= by).all(), f"{what}: off by {np.max(off / np.maximum(by, 1e-300))} of what it may be"


def check(lib, x, res, w, eps, form, rot=0, packed=False):
    y, z, r, h = plain.norm(x, res, w, eps)
    M, K = x.shape
    args = cuda(x, w, res)
    if form == "bf16":
        got, hg = lib.w8a8_rmsnorm(args[0], args[1], args[2], eps)
        close(plain.f64(got), y, np.abs(y) * (2.0 ** -8 + R_TOL) + 2.0 ** -133, "y")
    else:
        name = {"int8": "w8a8_rmsnorm_quantize", "fp8": "w8a8_rmsnorm_quantize_fp8", "block": "w8a8_rmsnorm_quantize_block"}[form]
        more = {} if form == "block" else dict(rot_block=rot)
        q, s, hg = getattr(lib, name + ("_packed" if packed else ""))(args[0], args[1], args[2], eps, **more)
        q, s = q.cpu().numpy(), s.cpu().numpy()
        if packed:
            q = plain.unpack(q, M, K)
            s = s[:, :M].T if form == "block" else s
        qmax = np.float32(127 if form == "int8" else 448)
        of = 128 if form == "block" else K
        codes_of = plain.int8_codes if form == "int8" else plain.e4m3_codes
        if not rot:
            v = z.astype(np.float32).reshape(-1, of)
            assert (v == z.reshape(-1, of)).all()                     # the products are fp32 values
            sz = np.abs(v).max(1) / qmax
            assert np.array_equal(q.reshape(-1, of).view(np.uint8), codes_of(v, sz).view(np.uint8)), "codes"
            want = sz.astype(np.float64).reshape(M, -1) * r
            close(s.astype(np.float64).reshape(M, -1), want, want * R_TOL, "scales")
        else:
            t = (y.reshape(-1, 128) @ plain.hadamard()).reshape(M, K)
            slack = np.repeat(np.abs(y).reshape(M, -1, 128).sum(-1), 128, axis=1) * ROT_TOL / 128 ** 0.5
            want = np.abs(t).max(1) / qmax
            close(s.astype(np.float64), want, want * R_TOL + slack.max(1) / qmax, "scales")
            by = s.astype(np.float64)[:, None]
            values = (q.astype(np.float64) if form == "int8" else plain.e4m3_values(q)) * by
            step = by if form == "int8" else np.maximum(np.abs(t) * 2.0 ** -3, by * 2.0 ** -9)   # E4M3: half a step is 2^-4 of the value
            close(values, t, step / 2 + (slack + np.abs(t) * R_TOL + want[:, None] * qmax * R_TOL), "rotated values")
    if res is None:
        assert hg is None
    else:
        assert torch.equal(hg.cpu(), h)


@pytest.mark.parametrize("M,K", ((1, 8), (3, 16), (1, 72), (2, 520), (5, 1024), (1, 5120), (300, 264), (257, 5120), (259, 2056),
                                 (2, 17408), (300, 8200), (1, 32776), (1, 65544), (2, 131072)))
@pytest.mark.parametrize("residual", (False, True))
def test_bf16(lib, M, K, residual):
    say(f"norm {M} x {K}, residual {residual}")
    x, res, w = inputs(M, K, M + K, residual)
    check(lib, x, res, w, 1e-6, "bf16")


@pytest.mark.parametrize("M,K", ((1, 32), (3, 96), (2, 1056), (33, 1024), (300, 5120), (1, 17408), (2, 131072)))
@pytest.mark.parametrize("form", ("int8", "fp8"))
def test_codes(lib, M, K, form):
    say(f"norm {M} x {K} {form}")
    x, res, w = inputs(M, K, 3 * M + K)
    check(lib, x, res, w, 1e-5, form)
    if K % 64 == 0:
        check(lib, x, None, w, 1e-5, form, packed=True)


@pytest.mark.parametrize("M,K", ((1, 128), (3, 384), (33, 1024), (300, 5120), (40, 17408), (1, 131072)))
@pytest.mark.parametrize("form", ("int8", "fp8", "block"))
def test_blocks_of_128(lib, M, K, form):
    """Rotated codes, and codes with a scale for each block."""
    say(f"norm {M} x {K} {form}, blocks of 128")
    x, res, w = inputs(M, K, 5 * M + K)
    rot = 0 if form == "block" else 128
    check(lib, x, res, w, 1e-6, form, rot, packed=True)
    check(lib, x, None, w, 1e-6, form, rot)


@pytest.mark.parametrize("form", ("bf16", "int8", "fp8", "block"))
def test_rows_of_zeros_and_far_from_one(lib, form):
    x, res, w = inputs(6, 256, 9)
    x[1], res[1] = 0, 0
    x[2] = x[2] * 2.0 ** 40
    x[3], res[3] = (x[3].float() * 2.0 ** -60).to(torch.bfloat16), 0
    x[4, 128:], res[4, 128:] = 0, 0
    x[5], res[5] = 0, 0
    x[5, 200] = -3.0
    check(lib, x, res, w, 1e-6, form)
    check(lib, x, res, w, 1e-30, form)


@pytest.mark.parametrize("form", ("bf16", "int8", "fp8", "block"))
def test_a_row_that_is_not_finite_spoils_itself_only(lib, form):
    x, res, w = inputs(5, 512, 10)
    clean = x.clone()
    x[1, 7], x[3, 500] = float("nan"), float("inf")
    f = {"bf16": lib.w8a8_rmsnorm, "int8": lib.w8a8_rmsnorm_quantize, "fp8": lib.w8a8_rmsnorm_quantize_fp8,
         "block": lib.w8a8_rmsnorm_quantize_block}[form]
    a, b = f(x.cuda(), w.cuda(), res.cuda()), f(clean.cuda(), w.cuda(), res.cuda())
    keep = torch.tensor([0, 2, 4], device="cuda")
    for u, v in zip(a, b):
        assert torch.equal(u[keep], v[keep])
    values = (a[0] if form == "bf16" else a[1]).float().cpu().reshape(5, -1)
    assert not torch.isfinite(values[1]).any() and not torch.isfinite(values[3]).all()


def test_in_place_rows_read_twice(lib):
    x, res, w = cuda(*inputs(3, 131072, 15))
    y, h = lib.w8a8_rmsnorm(x, w, res)
    for at in (0, 1):
        x2, r2 = x.clone(), res.clone()
        place = (x2, r2)[at]
        assert torch.equal(lib.w8a8_rmsnorm(x2, w, r2, h=place)[0], y) and torch.equal(place, h)
    x2, r2 = x.clone(), res.clone()
    lib.w8a8_rmsnorm(x2, w, r2, h=r2, out=x2)
    assert torch.equal(x2, y) and torch.equal(r2, h)
    lib.w8a8_rmsnorm(h, w, out=h)
    assert torch.equal(h, lib.w8a8_rmsnorm(lib.w8a8_rmsnorm(x, w, res)[1], w)[0])


def test_in_place_and_given_outputs(lib):
    x, res, w = cuda(*inputs(37, 640, 11))
    y, h = lib.w8a8_rmsnorm(x, w, res)
    r2, x2 = res.clone(), x.clone()
    out = lib.w8a8_rmsnorm(x2, w, r2, h=r2, out=x2)
    assert out[0] is x2 or out[0].data_ptr() == x2.data_ptr()
    assert torch.equal(x2, y) and torch.equal(r2, h)
    x3 = x.clone()
    assert torch.equal(lib.w8a8_rmsnorm(x3, w, res, h=x3)[0], y) and torch.equal(x3, h)
    g = torch.empty_like(x)
    assert torch.equal(lib.w8a8_rmsnorm(x, w, h=g)[1], x) and torch.equal(g, x)       # without a residual h is x
    q, s = torch.empty(37, 640, dtype=torch.int8, device="cuda"), torch.empty(37, device="cuda")
    got = lib.w8a8_rmsnorm_quantize(x, w, res, out=(q, s))
    assert got[0].data_ptr() == q.data_ptr() and got[1].data_ptr() == s.data_ptr()
    want = lib.w8a8_rmsnorm_quantize(x, w, res)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and torch.equal(want[2], h)


def test_padding_rows_stay(lib):
    """Packed codes and scales of 37 rows: what belongs to rows 37 to 63 is left as it was."""
    x, res, w = cuda(*inputs(37, 256, 12))
    q = torch.full((lib.packed_bytes(37, 256),), 0xAB, dtype=torch.uint8, device="cuda")
    s = torch.full((2, lib.block_scale_stride(37)), -7.0, device="cuda")
    lib.w8a8_rmsnorm_quantize_block_packed(x, w, res, out=(q, s))
    rows = plain.unpack(q.cpu().numpy(), 64, 256)
    assert (rows[37:] == 0xAB).all() and (s[:, 37:] == -7).all() and (s[:, :37] > 0).all()


def test_a_rows_result_does_not_depend_on_the_others(lib):
    """The same rows in calls of 3 and of 600, codes and scales (the sums' order goes by the number of rows, so scales may differ
    by their tolerance; codes may not)."""
    x, res, w = cuda(*inputs(600, 5120, 13))
    for f in (lib.w8a8_rmsnorm_quantize, lib.w8a8_rmsnorm_quantize_block):
        a, b = f(x, w, res), f(x[:3].contiguous(), w, res[:3].contiguous())
        assert torch.equal(a[0][:3], b[0]) and torch.equal(a[2][:3], b[2])
        assert ((a[1][:3] - b[1]).abs() <= b[1] * 2 * R_TOL).all()


def test_empty_and_refused(lib):
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    assert lib.w8a8_rmsnorm(x, w)[0].shape == (0, 64)
    assert lib.w8a8_rmsnorm_quantize(x, w)[0].shape == (0, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        with pytest.raises(lib.W8A8Error, match="BAD_ARGUMENT"):
            lib.w8a8_rmsnorm(x, w, **bad)
    with pytest.raises(lib.W8A8Error, match="BAD_ARGUMENT"):
        lib.w8a8_rmsnorm_quantize(x, w, rot_block=64)
    with pytest.raises(lib.W8A8Error, match="BAD_SHAPE"):
        lib.w8a8_rmsnorm_quantize(x, w, rot_block=128)
    with pytest.raises(lib.W8A8Error, match="BAD_SHAPE"):
        lib.w8a8_rmsnorm_quantize_block(x, w)
    with pytest.raises(ValueError, match="weight"):
        lib.w8a8_rmsnorm(x, w[:32].contiguous())
    with pytest.raises(ValueError, match="residual"):
        lib.w8a8_rmsnorm(x, w, x[:3].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        lib.w8a8_rmsnorm(x[:, ::2], w[:32].contiguous())
    with pytest.raises(TypeError):
        lib.w8a8_rmsnorm(x.float(), w)
    with pytest.raises(TypeError):
        lib.w8a8_rmsnorm(x, w, eps="small")
    with pytest.raises(ValueError, match="device"):
        lib.w8a8_rmsnorm(x.cpu(), w)
    with pytest.raises(ValueError, match="h: expected shape"):
        lib.w8a8_rmsnorm(x, w, x, h=x[:2].contiguous())


def test_captured_and_on_another_stream(lib):
    x, res, w = cuda(*inputs(70, 1024, 14))
    want = [t.clone() for t in lib.w8a8_rmsnorm_quantize_packed(x, w, res, rot_block=128)]
    bufs = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.w8a8_rmsnorm_quantize_packed(x, w, res, rot_block=128, h=bufs[2], out=(bufs[0], bufs[1]))
    M = 70
    for _ in range(3):
        for b in bufs:
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lib.unpack_rows(bufs[0], M, 1024), lib.unpack_rows(want[0], M, 1024))
        assert torch.equal(bufs[1], want[1]) and torch.equal(bufs[2], want[2])
