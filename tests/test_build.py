"""The library is built with or without its torch binding (a small source in the place of the kernels)."""
import ctypes
import os

import pytest

from fp8_scaled_gemm_sm_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int answer() { return 42; }\n')
    ext = tmp_path / "ext.cpp"
    ext.write_text("#include <torch/csrc/autograd/python_variable.h>\n#error does not compile\n")
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    for name, path in (("BUILD", "obj"), ("LIB", "lib.so"), ("EXT", "_ext.so"), ("EXT_SRC", "ext.cpp")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    return tmp_path


def _answers():
    return ctypes.CDLL(build.LIB).answer() == 42


def _without_torch(monkeypatch):
    import importlib.util

    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))

    def absent():
        raise ImportError("torch")

    monkeypatch.setattr(build, "_torch_dirs", absent)


def test_without_torch_the_library_alone_is_built(small, monkeypatch):
    _without_torch(monkeypatch)
    assert build.build() == build.LIB and _answers() and not os.path.exists(build.EXT)
    os.utime(build.LIB, (2 ** 31, 2 ** 31))  # newer than its sources: not built again
    assert build.up_to_date()


def test_a_binding_that_does_not_compile_leaves_the_library(small):
    with pytest.raises(RuntimeError, match="does not compile"):
        build.build()
    assert _answers() and not os.path.exists(build.EXT)
