"""The calls over a 4-bit cache, and the rotating append, on another stream than the
current one: what a call makes itself is made, and filled, on the stream it is given."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_469_b200 import lib
from tests import fp4_side

pytestmark = pytest.mark.gpu

WAIT = 100_000_000  # cycles: 50 ms and more of the current stream


def rows(tokens, hq=4, hkv=2, d=64):
    x = torch.randn(tokens, hq + 2 * hkv, d, device="cuda").bfloat16()
    return x.split([hq, hkv, hkv], 1)


def test_gather_on_a_stream_that_runs_ahead_of_the_current_one():
    rng = np.random.default_rng(1)
    tiles = fp4_side.random_tiles(rng, 6 * 2, 64).reshape(6, 2, 18 * 64)
    cache = torch.from_numpy(tiles).cuda()
    slots = torch.arange(0, 96, 3, device="cuda")
    want = lib.gather_fp4(cache, slots)
    given = torch.zeros_like(want[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    got = lib.gather_fp4(cache, slots, stream=side)
    half = lib.gather_fp4(cache, slots, k_out=given, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert want[0].any() and want[1].any()
    for pair in (got, half):
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


@pytest.mark.parametrize("make", ["append", "append4", "gather", "workspace"])
def test_new_memory_is_the_streams_own(make):
    """A tensor dropped on the current stream, whose work is still under way, is not
    what a call on another stream writes."""
    q, k, v = rows(512)
    slots = torch.arange(512, device="cuda")
    kc, vc = (torch.zeros(32, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = lib.new_fp4_cache(32, 2, 64)
    side = torch.cuda.Stream()
    call = {
        "append": lambda s: lib.rope_append(q, k, v, kc, vc, slots, None, None, stream=s),
        "append4": lambda s: lib.rope_append_fp4(q, k, v, cache, slots, None, None, stream=s),
        "gather": lambda s: lib.gather_fp4(cache, slots, stream=s)[0],
        "workspace": lambda s: lib.new_fp4_workspace(4, 40, 4, 2, 64, stream=s),
    }[make]
    like = call(None)
    torch.cuda.synchronize()
    del like
    held = [call(None) for _ in range(3)]
    torch.cuda.synchronize()
    taken = {t.data_ptr() for t in held}
    del held  # free again, on the current stream
    out = call(side)
    side.synchronize()
    assert out.data_ptr() not in taken


@pytest.mark.parametrize("which", ["k_out", "v_out"])
def test_gather_makes_the_output_that_is_not_given_like_the_other(which):
    tiles = fp4_side.random_tiles(np.random.default_rng(2), 4, 64).reshape(2, 2, 18 * 64)
    cache, slots = torch.from_numpy(tiles).cuda(), torch.arange(32, device="cuda")
    want = lib.gather_fp4(cache, slots, dtype=torch.float32)
    given = torch.zeros_like(want[0])
    got = lib.gather_fp4(cache, slots, **{which: given})
    assert given.data_ptr() in (got[0].data_ptr(), got[1].data_ptr())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
