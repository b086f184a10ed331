"""The library and the Python extension beside it are built apart: the library
does not need the interpreter's headers, and an extension belongs to the
interpreter that it was built for.  The compilers are stand-ins that write
empty files."""
import importlib.machinery
import os
import subprocess

import pytest

from bit_paged_kv_gb300 import build as B


@pytest.fixture
def ran(tmp_path, monkeypatch):
    """Programs run, in order; `ran.fail` names one that fails."""
    class Ran(list):
        fail = ()
    seen = Ran()

    def run(cmd, **kw):
        tool = os.path.basename(cmd[0])
        seen.append(tool)
        if tool in seen.fail:
            return subprocess.CompletedProcess(cmd, 1, "", "no such thing")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libsaw_int4.so"))
    monkeypatch.setattr(B, "STEP", str(tmp_path / os.path.basename(B.STEP)))
    return seen


def test_both_are_built_once(ran):
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and os.path.exists(B.STEP)
    n = len(ran)
    assert ran.count("g++") == 1 and n == len(B.UNITS) + 2
    B.build()
    assert len(ran) == n


def test_no_headers(ran, monkeypatch, tmp_path, capsys):
    """Without Python.h the library is built and the extension is not, nor is an old one left."""
    open(B.STEP, "w").close()
    os.utime(B.STEP, (1, 1))
    monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert not os.path.exists(B.STEP) and "g++" not in ran
    assert "no Python.h" in capsys.readouterr().err


def test_no_compiler(ran, monkeypatch):
    monkeypatch.setattr(B.shutil, "which", lambda name: None)
    assert B.build() == B.LIB and os.path.exists(B.LIB) and not os.path.exists(B.STEP)


def test_an_extension_that_does_not_compile_is_an_error_after_the_library(ran):
    ran.fail = ("g++",)
    with pytest.raises(RuntimeError, match="step_binding.cpp"):
        B.build()
    assert os.path.exists(B.LIB)


def test_another_interpreter_builds_its_own(ran, monkeypatch):
    """The file's name carries the interpreter's suffix; the library is not built again for another one."""
    assert os.path.basename(B.STEP) == "_saw_step" + importlib.machinery.EXTENSION_SUFFIXES[0]
    assert len(importlib.machinery.EXTENSION_SUFFIXES[0]) > len(".so")
    B.build()
    del ran[:]
    monkeypatch.setattr(B, "STEP", B.STEP.replace("_saw_step", "_saw_step.other"))
    B.build()
    assert ran == ["g++"]
