"""Which tile and how many parts of K a block product takes, on the CPU: that the shapes of tests/block_forms.py meet the forms that they are
meant for, all of them, and that parts never lack blocks."""
import ctypes
import shutil
import subprocess

import pytest

from block_forms import FORMS
from test_abi import LIB, ROOT
from test_sanitizers import ROCM

PROGRAM = r'''
#include <cstdio>
#include "block_choice.h"
using namespace w8a8::block_choice;
int main() {
  for (const Tile& t : kTiles) std::printf("tile %d %d\n", t.bm, t.bn);
  for (long long steps = 1; steps <= 128; steps *= 2)
    for (long long wide = 8; wide <= 1 << 20; wide *= 2)
      if (fused_fits(1, wide, 1024 * steps)) std::printf("fused %lld %lld\n", wide, steps);
  long long m, n, k;
  while (std::scanf("%lld %lld %lld", &m, &n, &k) == 3) {
    const Choice c = choose(m, n, k);
    std::printf("%lld %lld %lld %d %d %d\n", m, n, k, kTiles[c.tile].bm, kTiles[c.tile].bn, c.splits);
  }
}
'''


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None or not (ROCM / "include" / "hip").exists():
        pytest.skip("g++ or HIP's headers not available")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cpp").write_text(PROGRAM)
    res = subprocess.run(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM / 'include'}", f"-I{ROOT / 'w8a8_quantized_linear_amd' / 'csrc'}",
                          str(d / "choice.cpp"), "-o", str(d / "choice")], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-3000:]

    def ask(shapes):
        out = subprocess.run([str(d / "choice")], input="\n".join("%d %d %d" % s for s in shapes), capture_output=True, text=True, timeout=60)
        assert out.returncode == 0
        lines = [line.split() for line in out.stdout.splitlines()]
        fused = [tuple(map(int, line[1:])) for line in lines if line[0] == "fused"]
        tiles = [tuple(map(int, line[1:])) for line in lines if line[0] == "tile"]
        got = [tuple(map(int, line)) for line in lines if line[0].isdigit()]
        return tiles, [(g[:3], g[3:5], g[5]) for g in got], fused
    return ask


def test_every_form_is_met(ask):
    tiles, got, _ = ask([f[:3] for f in FORMS])
    assert got == [(f[:3], f[3], f[4]) for f in FORMS]
    assert {f[3] for f in FORMS if f[4] == 1} == set(tiles)
    assert {f[3] for f in FORMS if f[4] > 1} == set(tiles) - {(256, 256)}
    assert {f[4] for f in FORMS} == {1, 2, 3, 4, 6, 8, 12, 16}
    assert all(f[2] // 128 >= 9 for f in FORMS)              # more blocks of columns than stages in flight


def test_parts_have_blocks_and_a_workspace(ask):
    shapes = [(m, n, k) for m in (65, 84, 139, 330, 1502) for n in (8, 136, 1128, 4104, 16392) for k in (128, 1152, 2048, 4096, 13824, 131072)]
    lib = ctypes.CDLL(str(LIB))
    size = lib.w8a8_fp8_block_gemm_workspace_bytes
    size.restype, size.argtypes = ctypes.c_size_t, [ctypes.c_int64] * 3
    for (m, n, k), _, parts in ask(shapes)[1]:
        blocks = k // 128
        assert (parts - 1) * -(-blocks // parts) < blocks
        assert size(m, n, k) == (0 if parts == 1 else -(-4 * parts * m * n // 256) * 256)


def test_tokens_quantized_in_every_workgroup(ask):
    """Where each of eight waves has four steps of 128 columns at most; longer rows take a launch of their own, whatever the weight's rows."""
    fused = ask([])[2]
    assert {steps for _, steps in fused} == {1, 2, 4}
    assert {n for n, steps in fused if steps == 1} == {1 << i for i in range(3, 14)}
