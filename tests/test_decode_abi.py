"""Host-side checks of the few-token C entry points (no kernel is launched): sizes, refusals and their
order, on dummy pointers that are never dereferenced; and the same file's checks under the CPU sanitizers."""
import ctypes

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
    sig = {
        "w8a8_w4_code_bytes": (SZ, [I64, I64]),
        "w8a8_w4_scale_bytes": (SZ, [I64, I64, I]),
        "w8a8_w4_quantize": (I, [P, I64, I64, I, P, P, P]),
        "w8a8_w4_pack": (I, [P, P, I64, I64, I, P, P, P]),
        "w8a8_w4_workspace_bytes": (SZ, [I64, I64, I64]),
        "w8a8_w4_linear": (I, [P, P, P, P, P, I64, I64, I64, I, P, SZ, P]),
        "w8a8_kv_append": (I, [P, I64, P, I64, P, P, P, P, I64, P, I64, P] + [I64] * 5 + [P]),
        "w8a8_kv_read": (I, [P, P, P, P, I64, P, I64, P] + [I64] * 5 + [P, P, P]),
        "w8a8_kv_attention_workspace_bytes": (SZ, [I64] * 7),
        "w8a8_kv_attention": (I, [P, I64, P, P, P, P, I64, P, I64, P] + [I64] * 6 + [F, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def test_sizes(lib):
    assert lib.w8a8_w4_code_bytes(24, 256) == 32 * 128 and lib.w8a8_w4_code_bytes(0, 256) == 0
    assert lib.w8a8_w4_scale_bytes(24, 256, 64) == 32 * 4 * 2 and lib.w8a8_w4_scale_bytes(24, 256, 48) == 0
    ws = lib.w8a8_kv_attention_workspace_bytes
    assert ws(1, 1, 8, 8, 128, 64, 1) == 0                      # one piece of 128 tokens at most
    assert ws(1, 1, 8, 8, 128, 64, 1000) % 256 == 0 and ws(1, 1, 8, 8, 128, 64, 1000) > 0
    assert ws(4096, 1, 8, 8, 128, 64, 1000) == 0                # enough sequences: no pieces
    for bad in ((0, 1, 8, 8, 128, 64, 9), (1, 0, 8, 8, 128, 64, 9), (1, 1, 9, 8, 128, 64, 9), (1, 1, 8, 8, 96, 64, 9), (1, 1, 8, 8, 128, 64, 0)):
        assert ws(*bad) == 0


def test_w4_refusals(lib):
    def f(x, w, s, b, y, m, n, k, group, ws=A, ws_bytes=1 << 30):
        return lib.w8a8_w4_linear(x, w, s, b, y, m, n, k, group, ws, ws_bytes, None)

    assert f(A, A, A, None, A, -1, 16, 256, 64) == SHAPE
    assert f(A, A, A, None, A, (1 << 20) + 1, 16, 256, 64) == SHAPE
    assert f(A, A, A, None, A, 1, 12, 256, 64) == SHAPE
    assert f(A, A, A, None, A, 1, 0, 256, 64) == SHAPE
    assert f(A, A, A, None, A, 1, 16, 192, 64) == SHAPE
    assert f(A, A, A, None, A, 1, 16, 131072 + 128, 64) == SHAPE
    assert f(A, A, A, None, A, 1, 16, 256, 16) == BADARG
    assert f(None, None, None, None, None, 0, 16, 256, 64) == OK
    for i in (0, 1, 2, 4):
        p = [A, A, A, None, A]
        p[i] = None
        assert f(*p, 1, 16, 256, 64) == NULLP
        p[i] = U
        assert f(*p, 1, 16, 256, 64) == MISALIGNED
    assert f(A, A, A, U, A, 1, 16, 256, 64) == MISALIGNED
    need = lib.w8a8_w4_workspace_bytes(5, 1024, 16384)           # a long, narrow weight: K is cut
    assert need >= 2 * 5 * 1024 * 4 and need % 256 == 0
    assert f(A, A, A, None, A, 5, 1024, 16384, 64, A, need - 1) == BADARG
    assert f(A, A, A, None, A, 5, 1024, 16384, 64, None, need) == NULLP
    assert f(A, A, A, None, A, 5, 1024, 16384, 64, U, need) == MISALIGNED
    assert lib.w8a8_w4_workspace_bytes(5, 1024, 1024) == 0 and lib.w8a8_w4_workspace_bytes(0, 1024, 16384) == 0
    for g in (lambda n, k, grp, p=A: lib.w8a8_w4_quantize(p, n, k, grp, A, A, None),
              lambda n, k, grp, p=A: lib.w8a8_w4_pack(A, A, n, k, grp, p, A, None)):
        assert g(-1, 256, 64) == SHAPE and g(8, 192, 64) == SHAPE and g(8, 256, 7) == BADARG
        assert g(8, 256, 64, None) == NULLP and g(8, 256, 64, U) == MISALIGNED and g(0, 256, 64, None) == OK


def append(lib, **over):
    d = dict(k=A, ldk=256, v=A, ldv=256, kc=A, ks=A, vc=A, vs=A, pages=4, table=A, width=3, lens=A, seqs=2, tokens=5, heads=4, dim=64, page=16)
    return lib.w8a8_kv_append(*{**d, **over}.values(), None)


def attend(lib, **over):
    d = dict(q=A, ldq=512, kc=A, ks=A, vc=A, vs=A, pages=4, table=A, width=3, lens=A, seqs=2, tokens=5, q_heads=8, heads=4, dim=64, page=16,
             scale=0.125, y=A, ws=A, ws_bytes=1 << 30)
    return lib.w8a8_kv_attention(*{**d, **over}.values(), None)


def read(lib, **over):
    d = dict(kc=A, ks=A, vc=A, vs=A, pages=4, table=A, width=3, lens=A, seqs=2, length=9, heads=4, dim=64, page=16, k=A, v=A)
    return lib.w8a8_kv_read(*{**d, **over}.values(), None)


@pytest.mark.parametrize("call", (append, attend, read))
def test_cache_refusals(lib, call):
    for bad in (dict(seqs=-1), dict(heads=0), dict(heads=1025), dict(dim=96), dict(page=24), dict(page=256), dict(pages=0), dict(width=0),
                dict(width=(1 << 30) // 16 + 1), dict(seqs=(1 << 20) + 1)):
        assert call(lib, **bad) == SHAPE, bad
    for name in ("kc", "ks", "vc", "vs", "table", "lens"):
        assert call(lib, **{name: None}) == NULLP, name
        assert call(lib, **{name: U}) == MISALIGNED, name
    assert call(lib, seqs=0, kc=None, table=None) == OK


def test_append_refusals(lib):
    for bad in (dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(ldk=255), dict(ldk=248), dict(ldv=260), dict(seqs=1 << 20, tokens=1 << 20, heads=64, ldk=4096, ldv=4096)):
        assert append(lib, **bad) == SHAPE, bad
    for name in ("k", "v"):
        assert append(lib, **{name: None}) == NULLP and append(lib, **{name: U}) == MISALIGNED
    assert append(lib, tokens=0, k=None) == OK


def test_attention_refusals(lib):
    for bad in (dict(tokens=-1), dict(q_heads=6), dict(q_heads=2), dict(q_heads=2048, ldq=1 << 20), dict(ldq=504), dict(ldq=516),
                dict(seqs=1 << 20, tokens=1 << 20)):
        assert attend(lib, **bad) == SHAPE, bad
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert attend(lib, scale=scale) == BADARG
    need = lib.w8a8_kv_attention_workspace_bytes(2, 5, 8, 4, 64, 16, 300)
    assert need > 0 and attend(lib, width=300, ws_bytes=need - 1) == BADARG
    assert attend(lib, width=300, ws_bytes=need, ws=None) == NULLP and attend(lib, width=300, ws_bytes=need, ws=U) == MISALIGNED
    for name in ("q", "y"):
        assert attend(lib, **{name: None}) == NULLP and attend(lib, **{name: U}) == MISALIGNED
    assert attend(lib, tokens=0, q=None, ws=None, ws_bytes=0) == OK


def test_read_refusals(lib):
    for bad in (dict(length=-1), dict(length=(1 << 30) + 1), dict(seqs=1 << 20, length=1 << 30)):
        assert read(lib, **bad) == SHAPE, bad
    for name in ("k", "v"):
        assert read(lib, **{name: None}) == NULLP and read(lib, **{name: U}) == MISALIGNED
    assert read(lib, length=0, k=None) == OK


def test_valid_calls_without_a_gpu(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    assert lib.w8a8_w4_linear(A, A, A, A, A, 1, 16, 256, 64, None, 0, None) == DEVICE       # no workspace needed
    assert lib.w8a8_w4_quantize(A, 8, 256, 64, A, A, None) == DEVICE and lib.w8a8_w4_pack(A, A, 8, 256, 64, A, A, None) == DEVICE
    assert append(lib) == DEVICE and attend(lib) == DEVICE and read(lib) == DEVICE
    assert attend(lib, ws=None, ws_bytes=0, width=1) == DEVICE                # no workspace needed


def test_checks_under_asan_ubsan(tmp_path):
    """The host code of these entry points built with g++ under the sanitizers, at the ends of its ranges."""
    if not (ROCM / "lib" / "libamdhip64.so").exists():
        pytest.skip("HIP runtime not installed")
    import torch
    if torch.cuda.is_available():
        pytest.skip("the driver expects the no-device status that valid calls return without a GPU")
    csrc, san = ROOT / "w8a8_quantized_linear_amd" / "csrc", ROOT / "tests" / "sanitize"
    out = _build_and_run(tmp_path, "decode_abi_san",
                         [csrc / "api.cpp", csrc / "decode_api.cpp", san / "launcher_stubs.cpp", san / "decode_stubs.cpp",
                          san / "decode_abi_driver.cpp"],
                         ["-D__HIP_PLATFORM_AMD__", f"-I{ROCM / 'include'}", f"-I{ROOT / 'include'}", f"-I{csrc}",
                          f"-L{ROCM / 'lib'}", "-lamdhip64", f"-Wl,-rpath,{ROCM / 'lib'}"],
                         {"ASAN_OPTIONS": "detect_leaks=0"})
    assert "all argument checks as expected" in out
