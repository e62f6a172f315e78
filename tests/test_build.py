"""Building and loading the two binaries: the C library and the extension module
that marshals tensors into its serving calls (CPU only; no compiler runs here)."""
import os
import shutil
import sysconfig
import threading
import time

import pytest
import torch

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


def _copied_extension(monkeypatch, tmp_path):
    """A missing extension whose build copies the real one; returns the list of its builds."""
    real, builds = build_module.CALLS, []
    if not os.path.exists(real):
        build_module.build_calls()

    def build_calls():
        builds.append(threading.get_ident())
        time.sleep(0.2)
        shutil.copy(real, build_module.CALLS)
        return build_module.CALLS

    B.lib()
    monkeypatch.setattr(build_module, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build_module, "build_calls", build_calls)
    monkeypatch.setattr(B, "_CALLS", None)
    return builds


def test_threads_that_call_first_build_once(monkeypatch, tmp_path):
    builds, found = _copied_extension(monkeypatch, tmp_path), []
    threads = [threading.Thread(target=lambda: found.append(B._calls())) for _ in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(builds) == 1 and len(found) == 6 and all(m is found[0] for m in found)


def test_a_build_writes_to_a_file_of_its_process(monkeypatch):
    """Ranks that build at the same time do not write into each other's file."""
    commands = []

    class Failed:
        returncode, stderr = 1, "not run"

    monkeypatch.setattr(build_module.subprocess, "run", lambda cmd, **kw: commands.append(cmd) or Failed)
    with pytest.raises(RuntimeError, match="not run"):
        build_module.build_calls()
    out = commands[0][commands[0].index("-o") + 1]
    assert out != build_module.CALLS and str(os.getpid()) in os.path.basename(out)


def test_an_extension_of_another_torch_python_or_source_is_built_again(monkeypatch, tmp_path):
    """What is loaded was built from the present files against the present torch and Python."""
    if not build_module.calls_current():
        build_module.build_calls()
    assert build_module.calls_current()
    other = tmp_path / "torch_calls.cpp"
    other.write_text(open(build_module.CALLS_SRC).read() + "// changed")
    for change in ((torch, "__version__", "0.0"), (sysconfig, "get_config_var", lambda name: "cpython-00"),
                   (build_module, "CALLS_SRC", str(other)), (build_module, "BUILD", str(tmp_path))):
        with monkeypatch.context() as m:
            m.setattr(*change)
            assert not build_module.calls_current(), change
            m.setattr(B, "_CALLS", None)
            m.setattr(build_module, "build_calls", lambda: (_ for _ in ()).throw(RuntimeError("built again")))
            with pytest.raises(RuntimeError, match="built again"):
                B._calls()
    assert build_module.calls_current()


def test_an_extension_without_its_sources_is_taken_as_it_is(monkeypatch, tmp_path):
    """A package that was copied without its sources has nothing to build from."""
    extension = tmp_path / "_calls.so"
    monkeypatch.setattr(build_module, "CALLS", str(extension))
    monkeypatch.setattr(build_module, "CALLS_SRC", str(tmp_path / "torch_calls.cpp"))
    monkeypatch.setattr(build_module, "BUILD", str(tmp_path / "_build"))
    assert not build_module.calls_current()
    extension.touch()
    assert build_module.calls_current()
