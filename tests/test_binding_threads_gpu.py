"""Other Python threads run while a call of the module _binding is under way (a launch
blocks while the launch queue is full).  The library is a stand-in whose calls wait for
another thread; the tensors are on the GPU, nothing is launched there."""
from __future__ import annotations

import ctypes
import os
import subprocess
import threading
import time

import pytest
import torch

from paged_kv_cache_469_b200 import lib

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture
def stand_in(tmp_path):
    path = str(tmp_path / "libwaiting.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1",
                    os.path.join(HERE, "kernels", "waiting_library.c"), "-o", path], check=True)
    native = lib._marshal()
    native.load(path)
    try:
        yield ctypes.CDLL(path)
    finally:
        native.load(lib.LIB_PATH)


@pytest.mark.parametrize("which", ["append", "append4", "gather", "attention"])
def test_other_threads_run_during_a_call(stand_in, which):
    q, k = (torch.zeros(3, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(2, 2, 18 * 64, dtype=torch.uint8, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    i32 = torch.zeros(4, dtype=torch.int32, device="cuda")
    call = {
        "append": lambda: lib.rope_append(q, k, k, kc, kc, slots, None, None, q_out=q),
        "append4": lambda: lib.rope_append_fp4(q, k, k, cache, slots, None, None, q_out=q),
        "gather": lambda: lib.gather_fp4(cache, slots, k_out=k, v_out=k.clone()),
        "attention": lambda: lib.attention_varlen_fp4(
            torch.empty_like(q), q, cache, i32[:3].view(3, 1), i32[:3], i32, max_query_len=1,
            max_seq_len=16, scale=1.0, workspace=cache),
    }[which]
    go, waiting = (ctypes.c_int.in_dll(stand_in, name) for name in ("go", "waiting"))
    go.value = waiting.value = 0

    def other():
        while not waiting.value:
            time.sleep(0.001)
        go.value = 1
    thread = threading.Thread(target=other)
    thread.start()
    try:
        call()  # raises if nobody came in two seconds
    finally:
        waiting.value = 1
        thread.join()
