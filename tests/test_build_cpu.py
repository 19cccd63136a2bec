"""The build and the optional compiled module: the library stands without it, and a module of another ABI is not entered."""
import os
import re
import types

import pytest

import microscaling_fp4_quantized_amd as package
from microscaling_fp4_quantized_amd import binding
from microscaling_fp4_quantized_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_is_built_without_a_host_compiler(tmp_path, monkeypatch, capsys):
    lib, calls = tmp_path / "libfp4.so", tmp_path / "_torch_calls.so"
    calls.write_text("of an earlier build")
    for name, path in (("LIB", lib), ("CALLS", calls), ("BUILD", tmp_path / "objects")):
        monkeypatch.setattr(B, name, str(path))

    def none():
        raise RuntimeError("no host C++ compiler found")
    monkeypatch.setattr(B, "_compile", lambda src: src + ".o")
    monkeypatch.setattr(B, "_link", lambda objs: lib.write_text(" ".join(objs)))
    monkeypatch.setattr(B, "_build_calls", none)
    assert B.build() == str(lib)
    assert lib.read_text().split() == [s + ".o" for s in B.SOURCES]
    assert not calls.exists()
    assert "no host C++ compiler found" in capsys.readouterr().err


def test_a_library_that_does_not_build_is_an_error(tmp_path, monkeypatch):
    monkeypatch.setattr(B, "BUILD", str(tmp_path))

    def broken(src):
        raise RuntimeError("hipcc failed")
    monkeypatch.setattr(B, "_compile", broken)
    monkeypatch.setattr(B, "_build_calls", lambda: "")
    with pytest.raises(RuntimeError, match="hipcc failed"):
        B.build()


def functions():
    return {name: lambda *a: None for name in ("quantize", "norm", "linear", "route", "experts")}


@pytest.mark.parametrize("module,taken", [
    (types.SimpleNamespace(ABI_VERSION=None, **functions()), False),
    (types.SimpleNamespace(**functions()), False),
    (types.SimpleNamespace(ABI_VERSION="library's", **functions()), True)])
def test_a_module_of_another_abi_is_not_entered(module, taken, monkeypatch):
    if not os.path.exists(binding.library_path()):
        pytest.skip("libfp4.so not built")
    if binding._RAW_STREAM is None:
        pytest.skip("this torch has no raw stream handles")
    lib = binding.load_library()
    if getattr(module, "ABI_VERSION", None) == "library's":
        module.ABI_VERSION = lib.fp4_abi_version()
    monkeypatch.setattr(package, "_torch_calls", module, raising=False)
    assert bool(binding._compiled(lib)) == taken


def test_the_built_module_has_the_headers_version():
    if not os.path.exists(B.CALLS):
        pytest.skip("_torch_calls.so not built")
    from microscaling_fp4_quantized_amd import _torch_calls
    with open(os.path.join(ROOT, "include", "fp4.h")) as f:
        version = int(re.search(r"#define FP4_ABI_VERSION (\d+)", f.read()).group(1))
    assert _torch_calls.ABI_VERSION == version == binding.load_library().fp4_abi_version()
