"""What the build does when the Python module cannot be built (the C library does not
need it).  The library is linked from the objects of the build that is there."""
import ctypes
import os
import shutil
import sys

import pytest

from paged_kv_cache_469_b200 import build as b


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    b.build()
    shutil.copytree(b.BUILD, tmp_path / "_build")  # (times kept: nothing is compiled anew)
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libpa.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    return tmp_path


def loads(path):
    lib = ctypes.CDLL(path)
    lib.pa_status_string.restype = ctypes.c_char_p
    return bool(lib.pa_status_string(0))


def test_without_torch_the_library_is_built_alone(elsewhere, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # `import torch` fails
    assert b.build() == b.LIB and loads(b.LIB)
    assert not os.path.exists(b.BINDING)
    assert "_binding" in capsys.readouterr().err


def test_a_module_that_fails_leaves_the_library_and_says_so(elsewhere, monkeypatch):
    def fails(force):
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(b, "_binding", fails)
    with pytest.raises(RuntimeError, match="g.. failed"):
        b.build()
    assert loads(b.LIB)


def test_the_module_is_built_anew_for_another_torch(elsewhere, monkeypatch):
    import subprocess

    import torch
    ran = []

    def run(cmd, **kw):  # a compiler that writes its output at once
        ran.append(cmd[0])
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(b.subprocess, "run", run)
    b._binding(True)
    assert ran == ["g++"] and os.path.exists(b.BINDING)
    b._binding(False)
    assert ran == ["g++"], "nothing changed"
    monkeypatch.setattr(torch, "__version__", "0.0")
    b._binding(False)
    b._binding(False)
    assert ran == ["g++"] * 2
    os.utime(b.BINDING, (0, 0))  # older than its source
    b._binding(False)
    assert ran == ["g++"] * 3
