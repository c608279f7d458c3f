"""The order of the build, with stand-ins for the compilers: the C library
needs neither torch nor the binding."""

import os
import subprocess
import sys

import pytest

from host_paged_expert_gb300 import build


@pytest.fixture
def here(tmp_path, monkeypatch):
    """Compilers that write an empty output file; the commands that ran."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpe.so"))
    monkeypatch.setattr(build, "PYEXT", str(tmp_path / "_dense.so"))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def test_builds_both(here):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.PYEXT)


def test_library_without_torch(here, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.PYEXT)
    assert "torch is not installed" in capsys.readouterr().err


def test_library_before_a_binding_that_fails(here, monkeypatch):
    def fails():
        raise RuntimeError("compiling the binding failed")

    monkeypatch.setattr(build, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="binding"):  # said, not passed over
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.PYEXT)
