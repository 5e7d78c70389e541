"""libbq.so needs nvcc alone: the native form of the decoder-layer binding is an addition that the build and the calls
do without."""

import sys
import types

import pytest

torch = pytest.importorskip("torch")

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from quantized_mixed_precision_gb300 import build, decode  # noqa: E402


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A build whose compilers are stand-ins and whose outputs go to a folder of their own."""
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libbq.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_decode_binding.so"))
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "_compile", lambda src, extra: src)

    def run(cmd, **kw):
        if "-shared" in cmd and "g++" not in cmd[0]:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("lib")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build.subprocess, "run", run)
    return tmp_path


def test_a_binding_that_does_not_build_leaves_the_library(tree, monkeypatch):
    def fail():
        raise FileNotFoundError("g++")
    monkeypatch.setattr(build, "_build_binding", fail)
    (tree / "_decode_binding.so").write_text("of another torch")
    with pytest.warns(RuntimeWarning, match="g\\+\\+"):
        assert build.build() == build.LIB
    assert (tree / "libbq.so").exists()
    assert not (tree / "_decode_binding.so").exists()      # a stale one would be called with this library


def test_a_library_that_does_not_build_is_an_error(tree, monkeypatch):
    def fail(src, extra):
        raise RuntimeError("nvcc failed")
    monkeypatch.setattr(build, "_compile", fail)
    monkeypatch.setattr(build, "_build_binding", lambda: None)
    with pytest.raises(RuntimeError, match="nvcc"):
        build.build()


def test_calls_without_the_native_binding(monkeypatch):
    """The calls are bound and made from Python alone where the native form cannot be loaded."""
    name = "quantized_mixed_precision_gb300._decode_binding"
    monkeypatch.setitem(sys.modules, name, None)           # an import of it raises ImportError
    monkeypatch.delattr(bq, "_decode_binding", raising=False)
    monkeypatch.setattr(decode, "_bound", None)
    lib = types.SimpleNamespace(**{n: None for n in decode.SIGNATURES})
    monkeypatch.setattr(bq, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", None, raising=False)
    b = decode._load()
    assert b.native.gemm(1) is None and b.native.write() is None and b.native.attn(1, 2) is None
    with pytest.raises(TypeError):
        bq.bq_gemm_f16xi4_group(torch.zeros((1, 64)), None, None, 64)
