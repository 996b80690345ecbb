"""What the build needs of the machine: libdg only nvcc; the serving calls'
marshalling module gcc and Python's headers.  CPU only."""
import importlib.machinery
import os

import pytest

import fp16_tensor_core_gb300 as dg
from fp16_tensor_core_gb300 import build as dg_build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The marshalling module's file where none has been built."""
    native = os.path.join(tmp_path, os.path.basename(dg_build.NATIVE))
    monkeypatch.setattr(dg_build, "NATIVE", native)
    monkeypatch.setattr(dg, "_NATIVE_PATH", native)
    monkeypatch.setattr(dg, "_native", None)
    return native


@pytest.mark.parametrize("missing", ["Python.h", "gcc"])
def test_the_library_is_built_without_the_marshalling_module(monkeypatch, tmp_path, elsewhere, missing):
    if missing == "gcc":
        which = dg_build.shutil.which
        monkeypatch.setattr(dg_build.shutil, "which", lambda name: None if name == "gcc" else which(name))
    else:
        monkeypatch.setattr(dg_build.sysconfig, "get_paths", lambda: {"include": os.fspath(tmp_path)})
    with pytest.warns(UserWarning, match=missing):
        assert dg_build.build() == dg_build.LIB and os.path.exists(dg_build.LIB)
    assert dg.dg_gemm_plan(4096, 4096, 4096, sm_count=152)["grid"] > 0
    with pytest.raises(RuntimeError, match="not found; build it"):
        dg.dg_rope(None, None, None, None)


def test_errors_in_the_marshalling_module_are_errors(monkeypatch, tmp_path, elsewhere):
    (tmp_path / "dg_python.c").write_text("#error no\n")
    monkeypatch.setattr(dg_build, "CSRC", os.fspath(tmp_path))
    with pytest.raises(RuntimeError, match="gcc failed for dg_python.c"):
        dg_build._build_native(False)


def test_another_interpreter_loads_its_own(elsewhere):
    assert any(s != ".so" and elsewhere.endswith(s) for s in importlib.machinery.EXTENSION_SUFFIXES)
    assert os.path.basename(dg._NATIVE_PATH) == os.path.basename(dg_build.NATIVE)
    dg_build._build_native(False)
    assert os.path.exists(elsewhere) and dg._load_native().__file__ == elsewhere
