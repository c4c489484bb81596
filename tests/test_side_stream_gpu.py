"""The library's own side stream, of a step whose two kinds of work run on two streams,
while it is part of a capture: another mixed step on another stream meanwhile."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_469_b200 import lib
from tests.test_fp4_attention_gpu import Step

pytestmark = pytest.mark.gpu

QLS = [1] * 12 + [200] * 24
LENS = [8000] * 12 + [211] * 24


def four_bit(seed):
    st = Step(seed, LENS, QLS, 8, 2, 128, junk=False)
    return lambda out: st.run(host=True, out=out), torch.empty_like(st.q)


def bf16(seed):
    rng = np.random.default_rng(seed)
    lens, qsl = np.array(LENS, np.int32), np.concatenate([[0], np.cumsum(QLS)]).astype(np.int32)
    held = -(-lens // 16)
    tables = np.zeros((len(lens), int(held.max())), np.int32)
    order = rng.permutation(int(held.sum())).astype(np.int32)
    for s, n in enumerate(held):
        tables[s, :n], order = order[:n], order[n:]
    q, k, v = (torch.randn(*shape, device="cuda").bfloat16() for shape in
               ((int(qsl[-1]), 8, 128), *[(int(held.sum()), 2, 16, 128)] * 2))
    dev = [torch.from_numpy(x).cuda() for x in (tables, lens, qsl)]
    ws = lib.new_workspace(len(lens), 8, 2, 128, int(lens.max()))
    return (lambda out: lib.attention_varlen(
        out, q, k, v, *dev, max_query_len=200, max_seq_len=8000, scale=128 ** -0.5, workspace=ws,
        seq_lens_host=lens, query_start_loc_host=qsl)), torch.empty_like(q)


@pytest.mark.parametrize("kind", [four_bit, bf16])
def test_an_eager_mixed_step_while_one_is_captured(kind):
    (a, out_a), (b, out_b) = kind(1), kind(2)
    a(out_a), b(out_b)
    want = out_a.clone(), out_b.clone()
    other, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    out_a.fill_(float("nan")), out_b.fill_(float("nan"))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a(out_a)
        with torch.cuda.stream(other):
            b(out_b)
        a(out_a)
    torch.cuda.synchronize()
    close = dict(rtol=2.0 ** -7, atol=1e-3)  # (one after the other, the keys are cut otherwise)
    assert torch.isnan(out_a).all()
    torch.testing.assert_close(out_b, want[1], **close)
    graph.replay()
    assert torch.equal(out_a, want[0])
