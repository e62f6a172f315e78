"""Building and loading the two binaries: the C library and the extension module
that marshals tensors into its serving calls (CPU only; no compiler runs here)."""
import os

import pytest

from group_wise_affine_dequant_b200 import binding as B
from group_wise_affine_dequant_b200 import build as build_module


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The binaries' paths in an empty folder, linking by touching the file."""
    monkeypatch.setattr(build_module, "LIB", str(tmp_path / "libnvq.so"))
    monkeypatch.setattr(build_module, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build_module, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build_module, "_compile", lambda src, verbose: src)
    monkeypatch.setattr(build_module, "_link", lambda objs: open(build_module.LIB, "w").close())
    return tmp_path


def test_the_library_is_built_without_the_extension(elsewhere, monkeypatch):
    """A machine whose C++ compiler cannot build the extension still gets the C library, and an error that says so."""
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="false failed on"):
        build_module.build()
    assert os.path.exists(build_module.LIB) and not os.path.exists(build_module.CALLS)


def test_loading_the_library_builds_no_extension(elsewhere, monkeypatch):
    monkeypatch.setattr(build_module, "build_calls", lambda: pytest.fail("the extension is not needed"))
    monkeypatch.setattr(B, "_LIB", None)
    with pytest.raises(OSError):  # what the fixture links is no library
        B.lib()
    assert os.path.exists(build_module.LIB)
