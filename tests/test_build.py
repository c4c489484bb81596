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
