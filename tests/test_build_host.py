"""The build step: the C library alone where there is no PyTorch, and a binding
that was built for another PyTorch or Python is built again.  On a one-line library
and binding in a folder of their own."""
import ctypes
import os
import shutil
import sys

import pytest

CU = 'extern "C" int answer() { return 42; }\n'
CPP = '''#include <Python.h>
static PyModuleDef m = {PyModuleDef_HEAD_INIT, "_decode_ext", nullptr, -1, nullptr, nullptr, nullptr, nullptr, nullptr};
PyMODINIT_FUNC PyInit__decode_ext(void) { return PyModule_Create(&m); }
'''


@pytest.fixture
def small(tmp_path, monkeypatch):
    from sparse_spmv_memory_gb300 import _build
    (tmp_path / "a.cu").write_text(CU)
    (tmp_path / "binding.cpp").write_text(CPP)
    for name, value in dict(HERE=tmp_path, CSRC=tmp_path, INCLUDE=tmp_path / "include",
                            BUILD_DIR=tmp_path / "_build", LIB_PATH=tmp_path / "liba.so",
                            EXT_PATH=tmp_path / "_decode_ext.so", EXT_SOURCE=tmp_path / "binding.cpp").items():
        monkeypatch.setattr(_build, name, str(value))
    monkeypatch.setattr(_build, "SOURCES", ["a.cu"])
    if shutil.which(_build.nvcc()) is None and not os.path.exists(_build.nvcc()):
        pytest.skip("no nvcc")
    return _build


def test_the_library_is_built_without_pytorch(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # an import of it fails
    assert not small.up_to_date()
    path = small.build()
    assert ctypes.CDLL(path).answer() == 42
    assert not os.path.exists(small.EXT_PATH)
    assert small.up_to_date()
    made = os.path.getmtime(path)
    assert small.build() == path and os.path.getmtime(path) == made
    os.utime(os.path.join(small.CSRC, "a.cu"), (made + 5, made + 5))
    assert not small.up_to_date()


def test_a_binding_of_another_pytorch_is_built_again(small, monkeypatch):
    pytest.importorskip("torch")
    path = small.build()
    assert os.path.exists(small.EXT_PATH) and small.up_to_date()
    made, ext = os.path.getmtime(path), os.path.getmtime(small.EXT_PATH)
    real = small.importlib.metadata.version
    monkeypatch.setattr(small.importlib.metadata, "version", lambda name: real(name) + ".other")
    assert not small.up_to_date()
    os.utime(small.EXT_PATH, (ext - 5, ext - 5))
    small.build()
    assert os.path.getmtime(small.EXT_PATH) != ext - 5 and os.path.getmtime(path) == made
    assert small.up_to_date()
