"""The two parts of the build: libssd.so needs the CUDA toolkit only, so what
keeps the layer operators' binding from compiling must not keep it away."""
import ctypes
import os
import shutil

import pytest

from state_space_sequence_cumsum_gb300 import _build


@pytest.fixture
def small_tree(tmp_path, monkeypatch):
    """The build pointed at a library of one function and at a binding to come."""
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no CUDA toolkit")
    for name in ("csrc", "include"):
        (tmp_path / name).mkdir()
    (tmp_path / "csrc" / "one.cu").write_text('extern "C" int one(void) { return 1; }\n')
    for attr, path in (("CSRC", "csrc"), ("INCLUDE", "include"), ("BUILD", "_build"), ("LIB", "libssd.so"),
                       ("NATIVE", "_native.so"), ("BINDING", "csrc/binding.cpp"), ("PKG", "")):
        monkeypatch.setattr(_build, attr, os.fspath(tmp_path / path))
    return tmp_path


def test_library_without_its_binding(small_tree):
    (small_tree / "csrc" / "binding.cpp").write_text("#error no binding here\n")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        _build.build()
    assert ctypes.CDLL(_build.LIB).one() == 1
    assert _build.library_up_to_date() and not _build.binding_up_to_date() and not _build.up_to_date()
    with pytest.raises(RuntimeError, match="binding.cpp"):  # asked for again, refused again
        _build.build()


def test_binding_alone_is_rebuilt(small_tree):
    binding = small_tree / "csrc" / "binding.cpp"
    binding.write_text('extern "C" int one(void);\nextern "C" int two(void) { return one() + 1; }\n')
    _build.build()
    assert _build.up_to_date()
    built = os.path.getmtime(_build.LIB)
    os.utime(binding, (built + 10, built + 10))
    assert _build.library_up_to_date() and not _build.binding_up_to_date()
    os.utime(binding, (built - 10, built - 10))
    os.remove(_build.NATIVE)
    _build.build()
    assert _build.up_to_date() and os.path.getmtime(_build.LIB) == built
