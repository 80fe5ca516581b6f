"""The Python module of the plain calls (csrc/native.cpp) is extra: where it cannot be built or
loaded, the library is built all the same and the wrappers do all calls."""

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

import pytest
import torch

from jagged_gdpa_gb300 import _lib, build


@pytest.fixture
def own_calls(monkeypatch):
    """_lib as before its first native call."""
    build.build()
    monkeypatch.setattr(_lib, "_native", None)


def refuses_as_the_wrapper():
    four = [torch.zeros(4, 2, 16, n, dtype=t) for n, t in ((32, torch.uint8), (2, torch.bfloat16)) * 2]
    with pytest.raises(ValueError, match="CUDA device"):
        _lib.jgdpa_cache4_read(*four, torch.zeros(3, dtype=torch.int32))
    assert isinstance(_lib._native, _lib._NoNative)


def test_a_module_that_does_not_load(own_calls, monkeypatch, tmp_path):
    """Another interpreter's or another machine's file."""
    path = tmp_path / "_native.so"
    path.write_bytes(b"\x7fELF of another kind")
    monkeypatch.setattr(build, "native_path", lambda: str(path))
    with pytest.warns(RuntimeWarning, match="native calls"):
        refuses_as_the_wrapper()


def test_a_module_of_another_interface(own_calls, monkeypatch, tmp_path):
    """One that loads, but does not know this library's functions."""
    if not os.path.exists(build.native_path()):
        pytest.skip("no headers to build it from")
    monkeypatch.setattr(_lib, "EXPORTS", _lib.EXPORTS[:-1])
    with pytest.warns(RuntimeWarning, match="native calls"):
        refuses_as_the_wrapper()


def test_no_module(own_calls, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "native_path", lambda: str(tmp_path / "none.so"))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        refuses_as_the_wrapper()


def test_its_name_tells_what_it_was_built_for(monkeypatch, tmp_path):
    """torch, the interpreter's ABI, and the text of the header and the source: an older file is not taken."""
    path = build.native_path()
    assert torch.__version__ in path and sysconfig.get_config_var("SOABI") in path
    header = tmp_path / "jgdpa.h"
    header.write_text(open(build.HEADER).read() + "\n")
    monkeypatch.setattr(build, "HEADER", str(header))
    assert build.native_path() != path
    monkeypatch.undo()
    assert build.native_path() == path


def test_a_failed_compilation_leaves_the_library(monkeypatch, tmp_path):
    build.build()
    out = str(tmp_path / "never.so")
    monkeypatch.setattr(build, "_native_job", lambda cc, force: [sys.executable, "-c", "raise SystemExit('no such header')", out])
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert os.path.exists(build.build())
    assert not os.path.exists(build.native_path() + ".tmp") and not os.path.exists(out)


def test_builds_without_torch(tmp_path):
    """The C library's build needs no torch (here: up to date, so that nothing is compiled)."""
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no CUDA toolkit")
    build.build()
    (tmp_path / "torch.py").write_text("raise ImportError('not here')\n")
    r = subprocess.run([sys.executable, os.path.join(os.path.dirname(build.__file__), "build.py")], capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == build.LIB
