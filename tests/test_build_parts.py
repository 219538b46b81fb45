"""The library by itself: built without torch, and its package imported without the compiled part of the binding."""
import shutil
import subprocess
import sys

from test_abi import LIB, ROOT

PKG = ROOT / "w8a8_quantized_linear_amd"


def build_module():
    import __graft_entry__
    return __graft_entry__._hip_build_module()


def recorded(monkeypatch, tmp_path):
    """The build script with its compiler runs replaced: what it compiles and links, in order."""
    b, did = build_module(), []
    monkeypatch.setattr(b, "BUILD_DIR", tmp_path)
    monkeypatch.setattr(b, "_compile", lambda src, *a: tmp_path / src)
    monkeypatch.setattr(b, "_link", lambda objs, out: did.append(out.name))
    monkeypatch.setattr(b, "_link_binding", lambda obj: did.append("_binding.so"))
    return b, did


def test_without_torch_the_libraries_are_built_and_the_binding_is_left_out(monkeypatch, tmp_path, capsys):
    b, did = recorded(monkeypatch, tmp_path)
    monkeypatch.setitem(sys.modules, "torch", None)
    assert b.build() == b.LIB
    assert did == ["libw8a8.so", "libw8a8_probe.so"]
    assert "torch" in capsys.readouterr().err


def test_a_binding_that_does_not_compile_is_an_error_after_the_libraries(monkeypatch, tmp_path):
    b, did = recorded(monkeypatch, tmp_path)

    def fail():
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(b, "_compile_binding", fail)
    try:
        b.build()
    except RuntimeError as e:
        assert "g++ failed" in str(e)
    else:
        raise AssertionError("no error")
    assert did == ["libw8a8.so", "libw8a8_probe.so"]


def test_the_package_without_its_compiled_part(tmp_path):
    """Everything that goes through ctypes works; the few-token calls say what is missing."""
    if not LIB.exists():
        build_module().build()
    to = tmp_path / PKG.name
    to.mkdir()
    for name in ("__init__.py", "libw8a8.so"):
        shutil.copy(PKG / name, to / name)
    code = ("import w8a8_quantized_linear_amd as w8\n"
            "assert w8.__file__.startswith(%r)\n"
            "assert w8.packed_bytes(40, 128) == 64 * 128 and w8.w4_code_bytes(24, 256) == 32 * 128\n"
            "try:\n    w8.w8a8_w4_linear(None, None, None, 8, 64)\n"
            "except ImportError as e:\n    assert '_binding.so' in str(e) and 'build.py' in str(e), e\n"
            "else:\n    raise SystemExit('no error')\n" % str(tmp_path))
    res = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
