"""Host-side checks of the C entry points for norms, rotary positions and E4M3 projections with block scales (no kernel is
launched): sizes, refusals and their order, on dummy pointers that are never dereferenced; the same checks under the CPU
sanitizers; and the frequencies of rotary plans."""
import ctypes
import math

import pytest

from test_abi import A, BADARG, DEVICE, LIB, MISALIGNED, NULLP, OK, ROOT, SHAPE, U
from test_sanitizers import ROCM, _build_and_run

P, I64, I, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    if not LIB.exists():
        import __graft_entry__
        __graft_entry__._hip_build_module().build()
    lib = ctypes.CDLL(str(LIB))
    coded = (I, [P, P, P, F, I, P, P, P, I64, I64, P])
    block = (I, [P, P, P, F, P, P, P, I64, I64, P])
    sig = {
        "w8a8_rmsnorm": (I, [P, P, P, F, P, P, I64, I64, P]),
        "w8a8_rmsnorm_quantize": coded, "w8a8_rmsnorm_quantize_packed": coded,
        "w8a8_rmsnorm_quantize_fp8": coded, "w8a8_rmsnorm_quantize_fp8_packed": coded,
        "w8a8_rmsnorm_quantize_block": block, "w8a8_rmsnorm_quantize_block_packed": block,
        "w8a8_rope": (I, [P, I64, P, I64, P, I64, I, F, P] + [I64] * 5 + [P, I64, P, I64, P]),
        "w8a8_block_scale_stride": (I64, [I64]),
        "w8a8_quantize_act_block": (I, [P, I64, I64, P, P, P]), "w8a8_quantize_act_block_packed": (I, [P, I64, I64, P, P, P]),
        "w8a8_quantize_weight_block": (I, [P, I64, I64, P, P, P]),
        "w8a8_fp8_block_gemm_packed": (I, [P, P, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "w8a8_fp8_block_gemm_workspace_bytes": (SZ, [I64, I64, I64]), "w8a8_fp8_block_workspace_bytes": (SZ, [I64, I64, I64]),
        "w8a8_fp8_block_linear_packed": (I, [P, P, P, P, P, I64, I64, I64, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def gone():
    import torch
    return OK if torch.cuda.is_available() else DEVICE


def test_sizes(lib):
    assert [lib.w8a8_block_scale_stride(m) for m in (-1, 0, 1, 32, 33, 1 << 62)] == [0, 0, 32, 32, 64, 0]
    size, sums = lib.w8a8_fp8_block_workspace_bytes, lib.w8a8_fp8_block_gemm_workspace_bytes
    assert size(33, 16, 256) == 64 * 256 + 512 and sums(33, 16, 256) == 0
    for bad in ((0, 16, 256), (1, 16, 0), (1, 12, 256), (-5, 16, 256), (1, 16, 192)):
        assert size(*bad) == 0 and sums(*bad) == 0
    assert sums(100, 5120, 17408) % (100 * 5120 * 4) < 256 and sums(100, 5120, 17408) >= 2 * 100 * 5120 * 4   # few tiles, long K: parts
    assert sums(4096, 17408, 5120) == 0 and size(100, 5120, 17408) == 128 * 17408 + 136 * 512 + sums(100, 5120, 17408)


def test_norm_refusals(lib):
    def bf16(x=A, r=None, w=A, eps=1e-6, h=None, y=A, m=4, k=64):
        return lib.w8a8_rmsnorm(x, r, w, eps, h, y, m, k, None)

    assert bf16(m=-1) == SHAPE and bf16(m=(1 << 31) + 1) == SHAPE and bf16(k=0) == SHAPE and bf16(k=12) == SHAPE
    assert bf16(k=131072 + 8) == SHAPE
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert bf16(eps=eps) == BADARG
    assert bf16(m=0, x=None, w=None, y=None) == OK
    assert bf16(x=None) == NULLP and bf16(w=None) == NULLP and bf16(y=None) == NULLP
    for name in ("x", "r", "w", "h", "y"):
        assert bf16(**{name: U}) == MISALIGNED

    def coded(name, k=128, rot=0, q=A, s=A, m=4):
        return getattr(lib, name)(A, A, A, 1e-6, rot, A, q, s, m, k, None)
    for name in ("w8a8_rmsnorm_quantize", "w8a8_rmsnorm_quantize_fp8"):
        assert coded(name, k=48) == SHAPE and coded(name + "_packed", k=96) == SHAPE
        assert coded(name, rot=64) == BADARG and coded(name, k=96, rot=128) == SHAPE
        assert coded(name, q=None) == NULLP and coded(name, s=None) == NULLP and coded(name, s=U) == MISALIGNED
        assert coded(name, m=0, q=None) == OK
    for name in ("w8a8_rmsnorm_quantize_block", "w8a8_rmsnorm_quantize_block_packed"):
        f = getattr(lib, name)
        assert f(A, A, A, 1e-6, A, A, A, 4, 192, None) == SHAPE and f(A, A, A, 0.0, A, A, A, 4, 256, None) == BADARG
        assert f(A, A, A, 1e-6, A, A, None, 4, 256, None) == NULLP and f(A, A, A, 1e-6, A, U, A, 4, 256, None) == MISALIGNED
    if gone() == DEVICE:
        assert bf16() == DEVICE and coded("w8a8_rmsnorm_quantize") == DEVICE


def test_rope_refusals(lib):
    def f(q=A, ldq=512, k=A, ldk=512, turns=A, rotary=64, inter=0, amp=1.0, lens=A, seqs=2, tokens=3, q_heads=4, heads=2, dim=64, qo=A, ldqo=512,
          ko=A, ldko=512):
        return lib.w8a8_rope(q, ldq, k, ldk, turns, rotary, inter, amp, lens, seqs, tokens, q_heads, heads, dim, qo, ldqo, ko, ldko, None)

    for bad in (dict(seqs=-1), dict(seqs=(1 << 20) + 1), dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(seqs=1 << 20, tokens=1 << 11), dict(q_heads=0),
                dict(q_heads=1025, ldq=1 << 20, ldqo=1 << 20), dict(heads=-1), dict(heads=1025, ldk=1 << 20, ldko=1 << 20), dict(dim=8, rotary=8),
                dict(dim=72), dict(dim=272, rotary=272, ldq=2048, ldqo=2048, ldk=2048, ldko=2048), dict(rotary=80), dict(rotary=24), dict(rotary=0),
                dict(ldq=248), dict(ldq=260), dict(ldqo=255), dict(ldk=120), dict(ldko=127), dict(ldq=(1 << 40) + 8)):
        assert f(**bad) == SHAPE, bad
    for amp in (float("nan"), float("inf")):
        assert f(amp=amp) == BADARG
    assert f(ldqo=1024) == BADARG and f(ldko=1024) == BADARG                 # in place with another stride
    assert f(seqs=0, q=None, turns=None) == OK and f(tokens=0, lens=None) == OK
    for name in ("q", "k", "turns", "lens", "qo", "ko"):
        assert f(**{name: None}) == NULLP and f(**{name: U}) == MISALIGNED
    if gone() == DEVICE:
        assert f() == DEVICE and f(heads=0, k=None, ko=None, ldk=0, ldko=0) == DEVICE


def test_block_refusals(lib):
    for f in (lib.w8a8_quantize_act_block, lib.w8a8_quantize_act_block_packed, lib.w8a8_quantize_weight_block):
        assert f(A, -1, 128, A, A, None) == SHAPE and f(A, 4, 64, A, A, None) == SHAPE and f(A, 4, 192, A, A, None) == SHAPE
        assert f(A, 4, 131072 + 128, A, A, None) == SHAPE and f(A, 1 << 40, 128, A, A, None) == SHAPE
        assert f(None, 0, 128, None, None, None) == OK
        assert f(None, 4, 128, A, A, None) == NULLP and f(A, 4, 128, None, A, None) == NULLP and f(A, 4, 128, A, None, None) == NULLP
        assert f(U, 4, 128, A, A, None) == MISALIGNED and f(A, 4, 128, A, U, None) == MISALIGNED

    def gemm(q=A, s=A, w=A, sw=A, b=None, y=A, m=4, n=16, k=256, ws=None, size=0):
        return lib.w8a8_fp8_block_gemm_packed(q, s, w, sw, b, y, m, n, k, ws, size, None)

    def linear(x=A, w=A, sw=A, b=None, y=A, m=4, n=16, k=256, ws=A, size=1 << 20):
        return lib.w8a8_fp8_block_linear_packed(x, w, sw, b, y, m, n, k, ws, size, None)
    for f in (gemm, linear):
        for bad in (dict(m=-1), dict(m=(1 << 30) + 1), dict(n=0), dict(n=12), dict(n=1 << 28), dict(k=64), dict(k=192), dict(k=131072 + 128),
                    dict(m=1 << 20, n=(1 << 20) + 8)):
            assert f(**bad) == SHAPE, bad
        assert f(m=0, w=None, y=None) == OK
        for name in ("w", "sw", "y"):
            assert f(**{name: None}) == NULLP and f(**{name: U}) == MISALIGNED
        assert f(b=U) == MISALIGNED
    assert gemm(q=None) == NULLP and gemm(s=U) == MISALIGNED and linear(x=None) == NULLP and linear(ws=None) == NULLP and linear(ws=U) == MISALIGNED
    assert linear(size=lib.w8a8_fp8_block_workspace_bytes(4, 16, 256) - 1) == BADARG
    need = lib.w8a8_fp8_block_gemm_workspace_bytes(100, 5120, 17408)
    assert gemm(m=100, n=5120, k=17408, ws=A, size=need - 1) == BADARG and gemm(m=100, n=5120, k=17408, size=need) == NULLP
    assert gemm(m=100, n=5120, k=17408, ws=U, size=need) == MISALIGNED
    if gone() == DEVICE:
        assert gemm() == DEVICE and linear(size=lib.w8a8_fp8_block_workspace_bytes(4, 16, 256)) == DEVICE


STUBS = r'''
#include "entry.h"
#include "layer.h"
namespace w8a8 {
w8a8_status check_device() { return W8A8_ERR_UNSUPPORTED_DEVICE; }
hipError_t launch_norm(const Norm&, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_rope(const Rope&, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_quantize_block(const uint16_t*, int64_t, int64_t, bool, uint8_t*, float*, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_quantize_weight_block(const uint16_t*, int64_t, int64_t, uint8_t*, float*, hipStream_t) { return hipErrorUnknown; }
bool block_fused_fits(int64_t m, int64_t, int64_t) { return m == 1; }
hipError_t launch_block_fused(const uint16_t*, const uint8_t*, const float*, const uint16_t*, uint16_t*, int64_t, int64_t, int64_t, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_block_gemm(const uint8_t*, const float*, const uint8_t*, const float*, const uint16_t*, uint16_t*, int64_t, int64_t, int64_t,
                             float*, hipStream_t) { return hipErrorUnknown; }
size_t block_gemm_workspace(int64_t m, int64_t n, int64_t) { return (size_t)m * (size_t)n; }
}
'''

DRIVER = r'''
#include <cstdio>
#include <limits>
#include "w8a8.h"
#include "entry.h"
int main() {
  uint16_t* a = reinterpret_cast<uint16_t*>(0x10000);
  uint8_t* b = reinterpret_cast<uint8_t*>(a);
  int8_t* c = reinterpret_cast<int8_t*>(a);
  float* f = reinterpret_cast<float*>(a);
  const int64_t values[] = {std::numeric_limits<int64_t>::min(), -1, 0, 1, 7, 8, 16, 32, 64, 128, 1 << 20, (int64_t)1 << 31, (int64_t)1 << 40,
                            std::numeric_limits<int64_t>::max()};
  int64_t calls = 0;
  for (int64_t m : values)
    for (int64_t k : values) {
      const float eps = m % 3 ? 1e-6f : std::numeric_limits<float>::quiet_NaN();
      w8a8_rmsnorm(a, a, a, eps, a, a, m, k, nullptr);
      w8a8_rmsnorm_quantize(a, a, a, eps, 0, a, c, f, m, k, nullptr);
      w8a8_rmsnorm_quantize_packed(a, a, a, 1.0f, 128, a, c, f, m, k, nullptr);
      w8a8_rmsnorm_quantize_fp8(a, a, a, eps, 5, a, b, f, m, k, nullptr);
      w8a8_rmsnorm_quantize_fp8_packed(a, a, a, eps, 0, a, b, f, m, k, nullptr);
      w8a8_rmsnorm_quantize_block(a, a, a, eps, a, b, f, m, k, nullptr);
      w8a8_rmsnorm_quantize_block_packed(a, a, a, eps, a, b, f, m, k, nullptr);
      w8a8_quantize_act_block(a, m, k, b, f, nullptr);
      w8a8_quantize_act_block_packed(a, m, k, b, f, nullptr);
      w8a8_quantize_weight_block(a, m, k, b, f, nullptr);
      w8a8_block_scale_stride(m);
      for (int64_t n : values) {
        w8a8_fp8_block_gemm_packed(b, f, b, f, a, a, m, n, k, a, (size_t)-1, nullptr);
        w8a8_fp8_block_workspace_bytes(m, n, k);
        w8a8_fp8_block_linear_packed(a, b, f, a, a, m, n, k, a, (size_t)-1, nullptr);
        w8a8_rope(a, n, a, k, reinterpret_cast<uint64_t*>(a), 64, 0, 1.0f, reinterpret_cast<int32_t*>(a), m, n, 4, 2, 64, a, n, a, k, nullptr);
        w8a8_rope(a, 1024, a, 1024, reinterpret_cast<uint64_t*>(a), k, 1, 1.0f, reinterpret_cast<int32_t*>(a), 1, 1, m, n, k, a, 1024, a, 1024, nullptr);
        calls += 4;
      }
    }
  std::printf("%lld calls returned\n", (long long)calls);
  return 0;
}
'''


def test_checks_under_the_sanitizers(tmp_path):
    if not (ROCM / "lib" / "libamdhip64.so").exists():
        pytest.skip("HIP runtime not installed")
    (tmp_path / "stubs.cpp").write_text(STUBS)
    (tmp_path / "driver.cpp").write_text(DRIVER)
    csrc = ROOT / "w8a8_quantized_linear_amd" / "csrc"
    out = _build_and_run(tmp_path, "layer_san", [csrc / "layer_api.cpp", tmp_path / "stubs.cpp", tmp_path / "driver.cpp"],
                         ["-D__HIP_PLATFORM_AMD__", f"-I{ROCM / 'include'}", f"-I{ROOT / 'include'}", f"-I{csrc}",
                          f"-L{ROCM / 'lib'}", "-lamdhip64", f"-Wl,-rpath,{ROCM / 'lib'}"], {"ASAN_OPTIONS": "detect_leaks=0"})
    assert "calls returned" in out


# ------------------------------------------------------------ frequencies ----

@pytest.fixture(scope="module")
def package():
    import w8a8_quantized_linear_amd as package
    return package


def test_frequencies(package):
    f, a = package.rope_frequencies(8)
    assert a == 1.0 and f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)
    assert package.rope_frequencies(8, scaling="linear", factor=4.0)[0] == pytest.approx([v / 4 for v in f], rel=1e-14)
    ntk = package.rope_frequencies(8, scaling="ntk", factor=16.0)[0]
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(f[-1] / 16, rel=1e-12)      # the fastest kept, the slowest divided


def test_frequencies_by_wavelength(package):
    f, _ = package.rope_frequencies(128, base=500000.0)
    g, a = package.rope_frequencies(128, base=500000.0, scaling="wavelength", factor=8.0, original=8192)
    assert a == 1.0
    for v, w in zip(f, g):
        length = 2 * math.pi / v
        if length < 8192 / 4:
            assert w == v
        elif length > 8192:
            assert w == pytest.approx(v / 8, rel=1e-14)
        else:
            t = (8192 / length - 1) / 3
            assert w == pytest.approx((1 - t) * v / 8 + t * v, rel=1e-12) and v / 8 <= w <= v


def test_frequencies_by_index(package):
    """Pairs that make more than 32 turns over the original length are kept, those of less than one divided."""
    f, _ = package.rope_frequencies(128)
    g, a = package.rope_frequencies(128, scaling="yarn", factor=16.0, original=4096)
    assert a == pytest.approx(0.1 * math.log(16) + 1, rel=1e-14)
    for i, (v, w) in enumerate(zip(f, g)):
        turns = 4096 * v / (2 * math.pi)
        assert v / 16 * (1 - 1e-12) <= w <= v
        if turns > 32 * 10000 ** (2 / 128):
            assert w == v, i
        if turns < 10000 ** (-2 / 128):
            assert w == pytest.approx(v / 16, rel=1e-14), i
    assert all(x >= y for x, y in zip(g, g[1:]))


def test_a_plans_turns(package):
    plan = package.rope(64, device="cpu", interleaved=True)
    f, _ = package.rope_frequencies(64)
    assert plan.interleaved and plan.turns.shape == (32,)
    for t, v in zip(plan.turns.tolist(), f):
        assert t / 2 ** 64 * 2 * math.pi == pytest.approx(v, rel=1e-15)


@pytest.mark.parametrize("bad", (dict(rotary=7), dict(rotary=0), dict(rotary=8, scaling="other"), dict(rotary=8, factor=0.0, scaling="linear"),
                                 dict(rotary=8, base=-1.0), dict(rotary=8, scaling="wavelength", low=4.0, high=4.0)))
def test_refused_frequencies(package, bad):
    with pytest.raises(ValueError):
        package.rope_frequencies(**bad)
