"""The build (combine_counting_sort_gb300/_build.py) on a library of one small source: the C library needs nvcc
alone, and only what is out of date is built."""
import os
import sys

import pytest

from combine_counting_sort_gb300 import _build

BINDING = "#include <torch/csrc/autograd/python_variable.h>\nint unused;\n"


@pytest.fixture
def small(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text("extern \"C\" int one() { return 1; }\n")
    (csrc / "binding.cpp").write_text(BINDING)
    lib = tmp_path / "_lib"
    for name, value in (("CSRC", csrc), ("BUILD", tmp_path / "_build"), ("LIB_DIR", lib), ("LIB", lib / "libmoe.so"), ("BINDING", lib / "_binding.so")):
        monkeypatch.setattr(_build, name, str(value))
    return csrc


def test_the_library_is_built_where_the_binding_cannot_be(small, monkeypatch):
    (small / "binding.cpp").write_text("#error no such header\n")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING) and not _build.up_to_date()
    built = os.path.getmtime(_build.LIB)
    (small / "binding.cpp").write_text(BINDING)
    with monkeypatch.context() as m:   # no torch at all
        m.setitem(sys.modules, "torch", None)
        with pytest.raises(ImportError):
            _build.build()
    assert os.path.getmtime(_build.LIB) == built   # not built again
    assert _build.build() == _build.LIB
    assert os.path.exists(_build.BINDING) and os.path.getmtime(_build.LIB) == built and _build.up_to_date()


def test_only_what_is_out_of_date(small):
    _build.build()
    lib, binding = os.path.getmtime(_build.LIB), os.path.getmtime(_build.BINDING)
    os.utime(small / "binding.cpp", (binding + 2, binding + 2))
    assert not _build.up_to_date()
    _build.build()
    assert os.path.getmtime(_build.LIB) == lib and os.path.getmtime(_build.BINDING) > binding
