"""The library is built where the binding's helper cannot be: without g++, without Python's headers, without torch."""
import os
import subprocess
import sys

import pytest

from collective_communication_primitives_b200 import build as B


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """Compilers that only write the file they are asked for; g++ fails as `how` says."""
    ran, how = [], {}

    def run(cmd, check):
        ran.append(os.path.basename(cmd[0]))
        if cmd[0] == "g++" and "fails" in how:
            raise how["fails"]
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(cmd[0])

    monkeypatch.setattr(B.subprocess, "run", run)
    for name, path in (("LIB", "lib.so"), ("OBJ_DIR", "objects"), ("PKG", "")):
        monkeypatch.setattr(B, name, str(tmp_path / path))
    return ran, how


@pytest.mark.parametrize("fails", [subprocess.CalledProcessError(1, ["g++"]), FileNotFoundError("g++")])
def test_without_a_compiler_or_headers(tools, fails, capsys):
    ran, how = tools
    how["fails"] = fails
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.marshal_path())
    assert "not built" in capsys.readouterr().err
    n = len(ran)
    del how["fails"]
    assert B.build() == B.LIB and os.path.exists(B.marshal_path())  # it is made up for
    assert ran[n:] == ["g++"]


def test_without_torch(tools, monkeypatch):
    ran, _ = tools
    monkeypatch.setitem(sys.modules, "torch", None)
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert "g++" not in ran


def test_a_library_that_fails_is_an_error(tools, monkeypatch):
    monkeypatch.setattr(B, "_nvcc", lambda: "nvcc")
    real = B.subprocess.run

    def run(cmd, check):
        if cmd[0] == "nvcc":
            raise subprocess.CalledProcessError(1, cmd)
        real(cmd, check)

    monkeypatch.setattr(B.subprocess, "run", run)
    with pytest.raises(subprocess.CalledProcessError):
        B.build()


def test_without_a_torch_that_loads(tools, monkeypatch):
    ran, _ = tools

    def path():
        raise OSError("libcudart.so: cannot open shared object file")

    monkeypatch.setattr(B, "marshal_path", path)
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert "g++" not in ran
    assert B.build(force=True) == B.LIB
