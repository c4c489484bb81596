"""The fork and join of a step whose two kinds of work run on two streams: whatever call
fails, the caller's stream waits for what the side stream was given.  The CUDA calls are
stand-ins (no GPU needed)."""
import os
import subprocess

import pytest

from paged_kv_cache_469_b200.build import CSRC, NVCC

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("side") / "side_by_side_probe")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", CSRC, "-I", cuda,
                    os.path.join(HERE, "kernels", "side_by_side_probe.cpp"), "-o", out], check=True,
                   capture_output=True)
    return lambda failing: subprocess.run([out, failing], check=True, capture_output=True,
                                          text=True).stdout.split()


def test_both_are_queued_between_fork_and_join(probe):
    assert probe("none") == ["start", "wait", "aside", "here", "done", "join", "true"]


@pytest.mark.parametrize("failing,steps", [
    ("start", ["start"]),                                   # nothing on the side stream yet
    ("wait", ["start", "wait"]),
    ("aside", ["start", "wait", "aside", "done", "join"]),  # it may have queued a part
    ("here", ["start", "wait", "aside", "here", "done", "join"]),
    ("done", ["start", "wait", "aside", "here", "done"]),
    ("join", ["start", "wait", "aside", "here", "done", "join"]),
])
def test_a_failure_is_reported_and_what_was_queued_is_joined(probe, failing, steps):
    assert probe(failing) == steps + ["false"]
