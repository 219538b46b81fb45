"""Build ``libw8a8.so`` (the C-ABI library) for gfx950 with hipcc, and, where torch is installed,
the compiled part of its Python binding with the host compiler, in-tree.

    python w8a8_quantized_linear_amd/build.py

(run as a script: importing the package loads the library this produces).

Every HIP source is compiled with packed-fp32 instruction selection disabled
and the correctly rounded fp32 divide the quantizer relies on.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
LIB = PKG / "libw8a8.so"
BINDING = PKG / "_binding.so"      # the compiled part of the Python binding (needs torch's headers)
BUILD_DIR = PKG / "_build"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")
ARCH = "gfx950"
SOURCES = ["quantize.hip", "gemm.hip", "swiglu.hip", "short.hip", "scratch.hip", "api.cpp",
           "w4.hip", "kv_cache.hip", "attention.hip", "attention_prompt.hip", "decode_api.cpp"]
# Per-source flags.  The quantizer's fp64 matrix instructions (the rotation's
# cross-quarter transform) take the VGPR form: their results feed vector
# instructions, and results in accumulation registers would cost two copies per
# value and, at 12,016 x 17,408, the third wave per SIMD.
EXTRA = {"quantize.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}
# measurement aids for the benchmark and the design tests (not the library's C ABI)
PROBE_DIR = PKG / "probe"
PROBE_SOURCES = ["mfma_probe.hip", "fp8_contraction.hip", "f64_mfma_layout.hip", "stream_probe.hip",
                 "lds_probe.hip"]
PROBE_LIB = PROBE_DIR / "libw8a8_probe.so"

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _compile(src: str, folder: Path = CSRC, tag: str = "") -> Path:
    obj = BUILD_DIR / (tag + src.rsplit(".", 1)[0] + ".o")
    obj.unlink(missing_ok=True)
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC, *COMMON, *EXTRA.get(src, []), *lang, "-c", str(folder / src), "-o", str(obj)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "'-packed-fp32-ops' is not a recognized feature for this target (ignoring feature)"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip():
        print(err, file=sys.stderr)
    return obj


def _link(objs, out: Path) -> Path:
    tmp = out.with_suffix(".so.tmp")
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *map(str, objs), "-o", str(tmp)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    # every kernel launched from host code must have its stub in the library
    nm = subprocess.run(["nm", "--undefined-only", str(tmp)], capture_output=True, text=True)
    missing = [l for l in nm.stdout.splitlines() if "__device_stub__" in l]
    if nm.returncode != 0 or missing:
        raise RuntimeError("link produced a library with undefined kernel stubs:\n" + "\n".join(missing))
    os.replace(tmp, out)
    return out


def _compile_binding() -> Path:
    import sysconfig
    from torch.utils.cpp_extension import include_paths
    obj = BUILD_DIR / "binding.o"
    obj.unlink(missing_ok=True)
    includes = [*include_paths(), "/opt/rocm/include", sysconfig.get_paths()["include"], str(INCLUDE)]
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-DUSE_ROCM", "-D__HIP_PLATFORM_AMD__",
           *(f"-isystem{i}" for i in includes[:-1]), f"-I{INCLUDE}", "-c", str(CSRC / "binding.cpp"), "-o", str(obj)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{CXX} failed for binding.cpp:\n{res.stderr}")
    return obj


def _link_binding(obj: Path) -> None:
    from torch.utils.cpp_extension import TORCH_LIB_PATH
    tmp = BINDING.with_suffix(".so.tmp")
    cmd = [CXX, "-shared", str(obj), f"-L{PKG}", "-l:libw8a8.so", f"-L{TORCH_LIB_PATH}", "-lc10", "-lc10_hip", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{TORCH_LIB_PATH}", "-o", str(tmp)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, BINDING)


def build() -> Path:
    """Build libw8a8.so (the library), probe/libw8a8_probe.so (measurement aids) and _binding.so (the
    compiled part of the Python binding; left out without torch, which the library by itself does not need)."""
    BUILD_DIR.mkdir(exist_ok=True)
    jobs = [(src, CSRC, "") for src in SOURCES] + [(src, PROBE_DIR, "probe_") for src in PROBE_SOURCES]
    torch = importlib.util.find_spec("torch") is not None
    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        binding = ex.submit(_compile_binding) if torch else None
        objs = list(ex.map(lambda j: _compile(*j), jobs))
    _link(objs[:len(SOURCES)], LIB)
    _link(objs[len(SOURCES):], PROBE_LIB)
    if binding is None:
        print("torch is not installed: _binding.so is left out", file=sys.stderr)
    else:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build())
