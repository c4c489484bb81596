"""Calls over the 4-bit cache that are refused before anything is launched (CPU)."""
from __future__ import annotations

import pytest

from paged_kv_cache_469_b200 import lib as palib


@pytest.fixture(scope="module")
def L():
    from paged_kv_cache_469_b200.build import build
    build()
    return palib.library()


def gather(L, **kw):
    args = dict(ko=1 << 20, vo=2 << 20, kv=3 << 20, gk=1.0, gv=1.0, slots=16, n=3, hkv=2, d=64,
                bs=16, nb=4, dt=1, stream=None)
    args.update(kw)
    return L.pa_gather_fp4(*args.values())


@pytest.mark.parametrize("dtype,row", [(0, 512), (1, 256)])
def test_gather_outputs_that_overlap(L, dtype, row):
    """Three rows of two heads of 64 each, a cache of 4 blocks (4 * 2 * 1152 bytes)."""
    at = 1 << 20
    for bad in (dict(vo=at), dict(vo=at + 2 * row), dict(vo=at - 2 * row), dict(ko=3 << 20),
                dict(ko=(3 << 20) + 4 * 2304 - 16), dict(vo=(3 << 20) - 2 * row)):
        assert gather(L, dt=dtype, **bad) == palib.PA_ERR_INVALID, bad


def test_host_tensors_are_refused_by_name():
    """Also where the call makes an output of its own first, and on a machine without a
    GPU."""
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    kc, cache = torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 18 * 64, dtype=torch.uint8)
    slots = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: palib.rope_append(q, k, k, kc, kc, slots, None, None),
                 lambda: palib.rope_append_fp4(q, k, k, cache, slots, None, None),
                 lambda: palib.gather_fp4(cache, slots)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
