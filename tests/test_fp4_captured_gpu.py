"""Captured calls of pa_attention_varlen_fp4 with host copies, replayed over other
lengths of the same query tokens; which kernels each of them launches is read off the
captured graph."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.graph_side import Captured
from tests.test_fp4_attention_gpu import Step

pytestmark = pytest.mark.gpu


def set_lens(st, lens):
    st.lens = np.asarray(lens, np.int32)
    st.dev[1].copy_(torch.from_numpy(st.lens))


@pytest.mark.parametrize("hq,hkv,d,qls,lens,ctas,side", [
    (8, 2, 128, [200] * 24, [211 + 7 * i for i in range(24)], 1, False),  # an item to a CTA
    (6, 2, 64, [300] * 14, [301 + i for i in range(14)], 1, False),  # heads that do not pair up
    (8, 1, 128, [640], [700], 6, False),                             # keys cut, few tiles
    (8, 1, 128, [640], [6000], 6, False),                            # and many
    (3, 1, 64, [1300], [2900], 6, False),                            # heads that do not pair up
    (8, 2, 128, [200] * 24 + [1] * 12, [211] * 24 + [8000] * 12, 1, True),  # beside decodes
])
def test_replays_with_host_copies_follow_the_device_lengths(hq, hkv, d, qls, lens, ctas, side):
    lens = np.array(lens, np.int32)
    longest = np.minimum(lens * 2 + 1000, 9000).astype(np.int32)
    st = Step(hq + d + len(qls), longest, qls, hq, hkv, d, junk=False)
    out = torch.empty_like(st.q)
    set_lens(st, lens)
    st.run(host=True, out=out)  # (makes the side stream of a step of both kinds)
    st.check(out)
    call = Captured(lambda: st.run(host=True, out=out))
    prefill, = call.of("prefill_fp4_kernel")
    assert not call.of("prefill_plan_kernel")
    assert (prefill[2] > 1) == (ctas > 1) and prefill[2] <= ctas
    assert len(call.of("decode_fp4_kernel")) == side
    if side:  # on shares of the SMs
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert prefill[1] + call.of("decode_fp4_kernel")[0][1] == sms
    for now in (lens, longest, lens + 130, np.asarray(qls), longest):
        set_lens(st, now)
        out.fill_(float("nan"))
        call.replay()
        st.check(out)
