"""Which kernels steps over a 4-bit cache run on, read off the captured call, and the
cases that only some of them reach: chunks whose keys are cut over a cluster with fewer
key tiles than CTAs, heads that do not pair up."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.graph_side import Captured
from tests.test_fp4_attention_gpu import Step

pytestmark = pytest.mark.gpu

DECODE, PREFILL, PLAN = "decode_fp4_kernel", "prefill_fp4_kernel", "prefill_plan_kernel"


def captured(st, host, out):
    """The step's call, run once and captured."""
    st.run(host=host, out=out)
    return Captured(lambda: st.run(host=host, out=out))


@pytest.mark.parametrize("hq,hkv,d,lens,qls", [
    (16, 2, 64, [6000, 100], [300, 100]),
    (8, 1, 128, [9000, 130], [300, 120]),
    (3, 1, 64, [6000, 200], [700, 90]),      # heads that do not pair up, from here on
    (3, 1, 64, [6000, 129], [700, 129]),
    (4, 4, 64, [7777, 260], [900, 257]),
    (3, 1, 128, [9000, 110], [600, 100]),
    (5, 5, 128, [7777, 260], [900, 257]),
])
@pytest.mark.parametrize("host", [False, True])
def test_ctas_of_a_cluster_without_a_tile(hq, hkv, d, lens, qls, host):
    """A long chunk and a short one: the CTAs that share the long one's keys are more
    than the short one's tiles (of four or five kv-heads only with host copies: their
    items are counted by the step's bounds without)."""
    st = Step(sum(lens) + d, lens, qls, hq, hkv, d)
    out = torch.full_like(st.q, float("nan"))
    call = captured(st, host, out)
    prefill, = call.of(PREFILL)
    assert prefill[2] > (-(-lens[1] // 128) if host or hkv < 4 else 1)
    assert bool(call.of(PLAN)) != host
    st.check(out)
    want = out.clone()
    # a NaN or an infinity stays in its row
    st.q[qls[0] // 2, 1, 9], st.q[5, 0, 0] = float("nan"), float("inf")
    st.q[qls[0] + 7, 2, 1] = float("nan")
    call.replay()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[qls[0] // 2, 1] = bad[5, 0] = bad[qls[0] + 7, 2] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (3, 1, 64), (5, 5, 128)])
def test_cut_keys_of_unpaired_heads_in_a_graph_and_on_two_streams(hq, hkv, d):
    """Lengths known on the device only, their bounds far above them; a captured call as
    the lengths grow, and beside another step on a second stream."""
    st = Step(hq + d, [9000, 6000], [900, 300], hq, hkv, d, junk=False)
    full, short = st.lens.copy(), np.array([910, 300], np.int32)
    st.dev[1].copy_(torch.from_numpy(short))
    out = torch.full_like(st.q, float("nan"))
    call = captured(st, False, out)
    prefill, = call.of(PREFILL)
    assert prefill[2] > 1 and call.of(PLAN)
    for now in (short, np.array([2000, 6000], np.int32), full, short):
        st.lens = now
        st.dev[1].copy_(torch.from_numpy(now))
        out.fill_(float("nan"))
        call.replay()
        st.check(out)
    other = Step(hq + d + 1, [5000], [900], hq, hkv, d)
    got = [out, torch.empty_like(other.q)]
    assert captured(other, True, got[1]).of(PREFILL)[0][2] > 1
    want = [x.clone() for x in got]
    other.check(want[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in got:
        x.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (s, step) in enumerate(zip(streams, (st, other))):
            with torch.cuda.stream(s):
                step.run(host=bool(i), out=got[i])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (32, 4, 64), (24, 8, 128), (32, 2, 64),
                                      (12, 4, 128)])
def test_many_chunks_and_decodes_run_on_both_kernels(hq, hkv, d):
    """Chunks around the tiles of 128 queries and 128 keys, enough of them that each
    item has a CTA of its own, between decodes."""
    qls = [128, 129, 127, 256, 300, 1, 200, 131, 255, 1, 257, 140, 128, 384, 130, 190] * 2
    lens = [128, 129, 300, 511, 300, 77, 513, 640, 255, 900, 270, 141, 1024, 385, 131, 700] * 2
    st = Step(hq + d + 3, lens, qls, hq, hkv, d)
    for host in (False, True):
        out = torch.full_like(st.q, float("nan"))
        call = captured(st, host, out)
        assert call.of(DECODE) and call.of(PREFILL)[0][2] == 1
        st.check(out)


def test_what_runs_on_the_decode_kernel_alone():
    for dtype, qls in (("bf16", [1] * 40), ("bf16", [16] * 9), ("f32", [300, 1, 40])):
        st = Step(len(qls), [400] * len(qls), qls, 8, 2, 128, dtype)
        for host in (False, True):
            out = torch.empty_like(st.q)
            assert [k[0] for k in captured(st, host, out).kernels] == [DECODE]
            st.check(out)
