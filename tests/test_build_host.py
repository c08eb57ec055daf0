"""The build: the library does not need what only the direct binding needs."""
import os
import subprocess

import pytest


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module with its outputs under a folder of the test's and a
    compiler that writes its output file and nothing else."""
    from bwd_rms_norm_gb300 import build as b
    for name, at in (("BUILD_DIR", "objects"), ("LIB_PATH", "lib.so"),
                     ("BINDING_PATH", "binding.so")):
        monkeypatch.setattr(b, name, str(tmp_path / at))
    b.fails = ()

    def run(cmd, **kw):
        if os.path.basename(cmd[0]) in b.fails:
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    yield b
    del b.fails


def test_everything(build):
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.BINDING_PATH)


@pytest.mark.parametrize("how", ["compiler", "import"])
def test_without_what_the_binding_needs(build, monkeypatch, capsys, how):
    """The library is linked, an older binding does not stay beside it, and
    the reason is said."""
    open(build.BINDING_PATH, "w").close()
    if how == "compiler":
        build.fails = ("g++",)
    else:
        def missing():
            raise ImportError("no module named torch: No such file")
        monkeypatch.setattr(build, "_build_binding", missing)
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
    assert "No such file" in capsys.readouterr().err


def test_a_failed_library_is_an_error(build):
    build.fails = ("nvcc",)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()
