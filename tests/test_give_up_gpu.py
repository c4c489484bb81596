"""What a warp and a role of the kernels do as they give up a wait.

No input of the library reaches that path, so a probe kernel drives the functions of
``csrc/pa_wait.cuh`` that it is made of, on barriers of its own, with limits of 1 ms
and 200 ms: a warp leaves a wait together whatever its lanes saw, and a role that gives
up waits for what it has under way, but not for ever.
"""
import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "kernels", "give_up_probe.cu")
OUT = os.path.join(HERE, "_build", "libgive_up_probe.so")

LIMIT_NS = 1_000_000
OTHER_NS = 200_000_000
STATUS_WAIT_TIMEOUT = 1   # kStatusWaitTimeout


def _probe():
    from paged_kv_cache_469_b200.build import ARCH, CSRC, INCLUDE, NVCC
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    deps = [SRC, os.path.join(CSRC, "pa_wait.cuh"), os.path.join(CSRC, "pa_internal.cuh")]
    if not os.path.exists(OUT) or os.path.getmtime(OUT) < max(map(os.path.getmtime, deps)):
        tmp = OUT + f".tmp{os.getpid()}"
        subprocess.run([NVCC, *ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
                        "-I", CSRC, "-I", INCLUDE, SRC, "-o", tmp, "-lcudart"], check=True,
                       capture_output=True)
        os.replace(tmp, OUT)
    lib = ctypes.CDLL(OUT)
    lib.give_up_probe.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_ulonglong,
                                  ctypes.c_ulonglong, ctypes.c_int]
    lib.give_up_probe.restype = ctypes.c_int
    return lib


def _run(mode):
    lib = _probe()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    result = torch.full((34,), -1, dtype=torch.int32, device="cuda")
    assert lib.give_up_probe(status.data_ptr(), result.data_ptr(), LIMIT_NS, OTHER_NS, mode) == 0
    torch.cuda.synchronize()
    *lanes, aborted, us = result.tolist()
    return int(status.item()), lanes, aborted, us


def test_probe_builds():
    """The probe compiles against the library's wait header (no GPU needed)."""
    _probe()


@pytest.mark.gpu
def test_a_warp_leaves_a_wait_together():
    status, lanes, aborted, us = _run(0)
    assert lanes == [0] * 32, "half of the lanes saw their phase, and none may go on"
    assert status == STATUS_WAIT_TIMEOUT and aborted == 1 and us >= LIMIT_NS // 1000
    status, lanes, aborted, us = _run(1)
    assert lanes == [1] * 32 and status == 0 and aborted == 0 and us < LIMIT_NS // 1000


@pytest.mark.gpu
def test_a_role_that_gives_up_waits_for_its_own_work():
    status, _, aborted, us = _run(2)
    assert status == 0 and aborted == 1
    assert LIMIT_NS // 1000 <= us < OTHER_NS // 1000 // 4, "it ends though nothing arrives"
    status, _, aborted, us = _run(3)
    assert status == 0 and aborted == 1
    assert 50 <= us < OTHER_NS // 1000 // 4, "it ends with the arrival, not with the abort flag"
