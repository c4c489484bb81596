"""pa_attention_varlen_fp4 against fp64 attention over the cache's exact values."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_469_b200 import lib
from tests import fp4_side

pytestmark = pytest.mark.gpu


class Step:
    """A step over a random 4-bit pool.  ``junk``: slots that hold no token get
    all-one bytes (NaN scales)."""

    def __init__(self, seed, lens, qls, hq, hkv, d, dtype="bf16", spread=1.0, q_spread=1.0,
                 junk=True, extra_tokens=0):
        rng = np.random.default_rng(seed)
        lens, qls = np.asarray(lens, np.int32), np.asarray(qls, np.int32)
        held = -(-lens // 16)
        blocks = int(held.sum()) + 4
        order = rng.permutation(blocks).astype(np.int32)
        wide = max(1, int(held.max()))
        self.tables = np.full((len(lens), wide), -5, np.int32)
        pool = fp4_side.random_tiles(rng, blocks * hkv, d, spread).reshape(blocks, hkv, 18 * d)
        at = 0
        for s, n in enumerate(held):
            self.tables[s, :n] = order[at:at + n]
            at += n
            if junk and lens[s] % 16:
                for off in range(lens[s] % 16, 16):
                    for h in range(hkv):
                        fp4_side.put_row(pool[self.tables[s, n - 1], h], off, d, [15] * d,
                                         [255] * (d // 16), [15] * d, [255] * (d // 16))
        if junk:
            pool[order[at:]] = 255
        self.lens, self.pool = lens, pool
        self.qsl = np.concatenate([[0], np.cumsum(qls)]).astype(np.int32)
        t = int(self.qsl[-1]) + extra_tokens
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        q = torch.from_numpy((rng.standard_normal((t, hq, d)) * q_spread).astype(np.float32)).to(dt)
        self.q64 = q.double().numpy()
        self.q, self.cache = q.cuda(), torch.from_numpy(pool).cuda()
        self.dev = [torch.from_numpy(x).cuda() for x in (self.tables, self.lens, self.qsl)]
        self.scale = d ** -0.5
        self.k_scale, self.v_scale = 0.8, 1.7
        self.max_q, self.max_len = int(max(1, qls.max())), int(max(1, lens.max()))
        self.ws = lib.new_fp4_workspace(len(lens), t, hq, hkv, d)
        self.dtype = dtype

    def run(self, host=False, out=None, **kw):
        if out is None:
            out = torch.full_like(self.q, float("nan"))
        args = dict(max_query_len=self.max_q, max_seq_len=self.max_len, scale=self.scale,
                    workspace=self.ws, k_scale=self.k_scale, v_scale=self.v_scale,
                    seq_lens_host=self.lens if host else None,
                    query_start_loc_host=self.qsl if host else None)
        return lib.attention_varlen_fp4(out, self.q, self.cache, *self.dev, **{**args, **kw})

    def check(self, out):
        rows = int(self.qsl[-1])
        want, mass, reach = fp4_side.attention(self.q64[:rows], self.pool, self.tables, self.lens,
                                               self.qsl, self.scale, self.k_scale, self.v_scale)
        got = out[:rows].double().cpu().numpy()
        d, n = want.shape[-1], float(self.lens.max())
        half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -24
        # a probability: rounded to f16 (two of them for fp32), its exponential
        # and the sums of up to n terms in fp32 (blocked: far fewer in a row
        # than n; sqrt(n) covers them), its score's error: up to D products and
        # sums of fp32 and the split query
        score = (d + 8) * 2.0 ** -24 * (1 + reach)
        p_half = 2.0 ** -11 if self.dtype == "bf16" else 2.0 ** -21
        rel = p_half + 2.0 ** -20 + np.sqrt(n) * 2.0 ** -23 + 2 * score
        vmax = 2 * np.abs(fp4_side.E2M1).max() * 8 * self.v_scale
        bound = half * np.abs(want) + rel[..., None] * 1.01 * mass + n * 2.0 ** -32 * vmax
        worst = np.max(np.abs(got - want) / bound) if want.size else 0.0
        assert np.isfinite(got).all() and worst <= 1.0, f"{worst:.3f} of the bound"
        head = self.ws[:256 + 1024].cpu()
        assert not head.any(), "the workspace header and counters are zero between calls"
        return worst


SHAPES = [(32, 8, 128), (32, 4, 64), (4, 4, 64), (8, 1, 128), (16, 1, 128), (16, 1, 64),
          (6, 2, 64), (7, 1, 128)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_steps(hq, hkv, d, dtype):
    st = Step(d + hq, [1, 2, 15, 16, 17, 31, 33, 100, 517, 1203], [1] * 10, hq, hkv, d, dtype)
    a = st.run()
    st.check(a)
    assert torch.equal(a, st.run(host=True)) and torch.equal(a, st.run())


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_several_query_tokens(hq, hkv, d, dtype):
    st = Step(2 * d + hq, [1, 5, 16, 40, 3, 300, 0, 129, 64], [1, 5, 2, 9, 0, 7, 0, 16, 3], hq, hkv,
              d, dtype)
    a = st.run()
    st.check(a)
    assert torch.equal(a, st.run(host=True))


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (32, 4, 64), (3, 1, 128), (8, 1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,qls", [([130], [130]), ([700, 65, 1], [257, 65, 1]),
                                      ([400, 20, 999, 300], [128, 1, 200, 129])])
def test_prompt_chunks(hq, hkv, d, dtype, lens, qls):
    st = Step(sum(lens) + d, lens, qls, hq, hkv, d, dtype)
    a = st.run()
    st.check(a)
    st.check(st.run(host=True))


def tensor_core_work(qls, lens, hq, hkv, d):
    """(ns of the chunks on the prefill kernel, ns on the decode kernel), by the rates
    that the library chooses with."""
    block_ns, tile_ns = (0.60, 1950.0) if d == 128 else (0.34, 1800.0)
    group = hq // hkv
    tiles = decode = longest = 0.0
    for q, n in zip(qls, lens):
        qt = -(-q // 128)
        items = qt * hq / 2 if group % 2 == 0 else -(-qt // 2) * hq
        tiles += items * -(-n // 128)
        longest = max(longest, -(-n // 128))
        decode += -(-n // 16) * -(-q * group // 16) * hkv * block_ns
    return max(tiles / 148, longest) * tile_ns, decode


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (32, 4, 64), (24, 8, 128), (32, 2, 64)])
def test_chunks_on_the_tensor_cores(hq, hkv, d):
    """Enough chunks that they run on the prefill kernel: lengths around its tiles of
    128 queries and 128 keys, with and without context, between decodes."""
    qls = [128, 129, 127, 256, 300, 1, 200, 131, 255, 1, 257, 140, 128, 384, 130, 190]
    lens = [128, 129, 300, 511, 300, 77, 513, 640, 255, 900, 270, 141, 1024, 385, 131, 700]
    chunks = [(q, n) for q, n in zip(qls, lens) if q > 1]
    tensor, decode = tensor_core_work(*zip(*chunks), hq, hkv, d)
    assert tensor + 16000 < decode, "the case is too small to reach the prefill kernel"
    st = Step(hq + d, lens, qls, hq, hkv, d)
    out = st.run(host=True)
    st.check(out)
    st.check(st.run())  # lengths known on the device only
    assert torch.equal(st.run(host=True), out)
    # a NaN or an infinity stays in its row
    st.q[300, 3, 9], st.q[5, 1, 0] = float("nan"), float("inf")
    got = st.run(host=True)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[300, 3] = bad[5, 1] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], out[~bad])
    # query rows behind the last sequence (without host copies, which would refuse them)
    st = Step(hq + d, lens, qls, hq, hkv, d, extra_tokens=2)
    out = torch.full_like(st.q, 9.0)
    st.run(out=out)
    st.check(out)
    assert (out[-2:] == 9.0).all()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("lens", [[20011], [9000, 3, 12000], [16 * 148 * 16], [16 * 148 * 16 + 1]])
def test_long_contexts_over_many_processors(hq, hkv, d, lens):
    st = Step(lens[0] + d, lens, [1] * len(lens), hq, hkv, d, junk=False)
    a = st.run()
    st.check(a)
    for _ in range(3):
        assert torch.equal(a, st.run())


@pytest.mark.parametrize("hq,hkv,d,lens,qls", [
    (8, 1, 128, [9000], [640]),              # 20 items of 71 tiles: four CTAs each
    (32, 8, 128, [5000], [512]),             # 64 items: two
    (4, 2, 128, [3001], [700]),              # 12: eight
    (4, 4, 64, [7777], [600]),               # heads that do not pair up, D = 64
    (3, 1, 64, [4000, 77], [513, 40]),       # and a short chunk's items beside: some
    (16, 2, 64, [6000, 600], [300, 600]),    # of a cluster's CTAs have no tile
])
def test_chunks_whose_keys_are_cut(hq, hkv, d, lens, qls):
    st = Step(sum(lens) + d, lens, qls, hq, hkv, d)
    a = st.run()
    st.check(a)
    b = st.run(host=True)
    st.check(b)
    assert torch.equal(a, st.run()) and torch.equal(b, st.run(host=True))
    # a NaN or an infinity stays in its row
    st.q[qls[0] // 2, 1, 9], st.q[5, 0, 0] = float("nan"), float("inf")
    got = st.run(host=True)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[qls[0] // 2, 1] = bad[5, 0] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], b[~bad])


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (4, 4, 64), (8, 2, 64)])
def test_cut_keys_follow_the_device_lengths(hq, hkv, d):
    """Bounds far above the lengths: more CTAs share a chunk's keys than it has tiles.
    The same captured call, as the lengths grow, and on two streams at once."""
    lens = np.array([300, 140], np.int32)
    st = Step(hq + d, [9000, 6000], [256, 129], hq, hkv, d, junk=False)
    full = st.lens.copy()
    st.dev[1].copy_(torch.from_numpy(lens))
    graph, out = torch.cuda.CUDAGraph(), torch.full_like(st.q, float("nan"))
    with torch.cuda.graph(graph):
        st.run(out=out)
    for now in (lens, np.array([2000, 6000], np.int32), full, lens):
        st.lens = now
        st.dev[1].copy_(torch.from_numpy(now))
        out.fill_(float("nan"))
        graph.replay()
        st.check(out)
    other = Step(hq + d + 1, [5000], [200], hq, hkv, d)
    want = [out.clone(), other.run()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [torch.full_like(w, float("nan")) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, step, o in zip(streams, (st, other), got):
            with torch.cuda.stream(s):
                step.run(out=o)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hq,hkv,d,lens,qls", [
    (16, 1, 128, [8727] * 5, [1] * 5),                # 30 processors a unit
    (8, 1, 64, [8270, 33083], [1, 1]),                # 30 and 118
    (16, 1, 64, [9000, 21000, 5], [4, 2, 1]),         # several units of one sequence
    (8, 1, 128, [40000], [1]),                        # all of them
    (7, 1, 64, [7300, 6900], [3, 3]),                 # about the size joined at once
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_units_over_many_processors(hq, hkv, d, lens, qls, dtype):
    st = Step(sum(lens) + d, lens, qls, hq, hkv, d, dtype)
    a = st.run()
    st.check(a)
    assert torch.equal(a, st.run(host=True)) and torch.equal(a, st.run())
    assert not st.ws[:256 + 3 * 1024].cpu().any(), "all arrival counters are zero between calls"


@pytest.mark.parametrize("lens,qls", [([300, 45, 517], [1, 200, 2]),  # (45: left out, its rows stay)
                                      ([300, 245, 517], [1, 200, 2]),
                                      ([400] * 24, [250] * 24)])  # (on the tensor cores)
def test_offsets_past_32_bits(lens, qls):
    """Blocks on both sides of 2 GB and 4 GB of a pool."""
    st = Step(31, lens, qls, 8, 8, 128, junk=False)
    want = st.run()
    blocks = (9 << 29) // (8 * 18 * 128)  # 4.5 GB
    rng = np.random.default_rng(2)
    far = np.sort(rng.choice(blocks, st.pool.shape[0], replace=False)).astype(np.int32)
    far[-1] = blocks - 1
    big = torch.empty(blocks, 8, 18 * 128, dtype=torch.uint8, device="cuda")
    big[torch.from_numpy(far).long().cuda()] = st.cache
    st.cache = big
    st.dev[0] = torch.from_numpy(np.where(st.tables >= 0, far[st.tables], -5)).int().cuda()
    assert torch.equal(st.run().view(torch.int16), want.view(torch.int16))
    slots = torch.from_numpy(far[::7].astype(np.int64) * 16 + 5).cuda()
    k, v = lib.gather_fp4(big, slots, dtype=torch.float32)
    kw, vw = fp4_side.tile_values(st.pool[::7], 128)
    assert np.array_equal(k.cpu().numpy(), kw[:, :, 5].astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), vw[:, :, 5].astype(np.float32))
    # rows appended there are found again
    x = torch.randn(len(slots), 8, 128, device="cuda").bfloat16()
    lib.rope_append_fp4(x[:, :0], x, x, big, slots, None, None)
    small = lib.new_fp4_cache(len(slots), 8, 128)
    lib.rope_append_fp4(x[:, :0], x, x, small, torch.arange(len(slots), device="cuda") * 16 + 5,
                        None, None)
    got = big[torch.from_numpy(far[::7]).long().cuda()]
    keep = small != 0
    assert torch.equal(got[keep], small[keep])


def test_two_graphs_share_a_workspace():
    """Two captured steps of different shape on one workspace, replayed in turn on one
    stream, with an eager step between."""
    a = Step(41, [3000, 200], [1, 1], 8, 2, 128)
    b = Step(42, [90, 400, 17], [70, 400, 17], 8, 2, 128)
    ws = lib.new_fp4_workspace(3, 487, 8, 2, 128)
    a.ws = b.ws = ws
    wants, graphs, outs = [], [], []
    for st in (a, b):
        wants.append(st.run())
        outs.append(torch.empty_like(st.q))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.run(out=outs[-1])
        graphs.append(g)
    for i in (0, 1, 1, 0, 0):
        outs[i].fill_(float("nan"))
        graphs[i].replay()
        assert torch.equal(outs[i], wants[i])
        assert torch.equal(b.run(host=True), wants[1])
    a.check(outs[0])


def test_a_nan_query_stays_in_its_row():
    for dtype in ("bf16", "f32"):
        st = Step(12, [150, 700], [100, 1], 8, 2, 64, dtype)
        want = st.run()
        st.q[5, 3, 7] = float("nan")
        st.q[100, 2, 0] = float("inf")
        got = st.run()
        bad = torch.zeros_like(got, dtype=torch.bool)
        bad[5, 3] = True
        bad[100, 2] = True
        assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,qls", [([4000, 70], [1, 1]), ([1300, 900], [9, 1]),
                                      ([1500] * 9, [300] + [512] * 8)])
def test_a_nan_in_the_cache_reaches_the_rows_that_see_it(lens, qls, dtype):
    """Also where a whole part of a sequence's keys holds nothing else; the rows that
    do not see it, the other heads' and the other sequences' stay as they were."""
    hq, hkv, d = 8, 2, 128
    st = Step(sum(lens), lens, qls, hq, hkv, d, dtype)
    want, pool = st.run(), st.pool.copy()
    first, last = lens[0] - qls[0] // 2 - 500, lens[0] - qls[0] // 2
    sees = torch.arange(st.qsl[-1]) >= qls[0] + first - lens[0]
    sees[qls[0]:] = False
    for tok in range(first, last):  # K of head 1
        tile = pool[st.tables[0, tok // 16], 1]
        tile[16 * d + tok % 16 * (d // 16):][:d // 16] = 127
    st.cache.copy_(torch.from_numpy(pool))
    got = st.run()
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[sees, 4:] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])

    pool = st.pool.copy()
    for tok in range(first, last):  # V of head 0, dims 32 .. 47
        pool[st.tables[0, tok // 16], 0, 17 * d + 2 * 16 + tok % 16] = 127
    st.cache.copy_(torch.from_numpy(pool))
    got = st.run()
    assert torch.isnan(got[sees, :4, 32:48]).all()
    kept = torch.ones_like(got, dtype=torch.bool)
    kept[:qls[0], :4, 32:48] = False
    assert torch.equal(got[kept], want[kept])


def test_a_prefix_shared_by_sequences_and_repeated_blocks():
    st = Step(13, [400, 400, 64], [1, 90, 1], 8, 2, 128, junk=False)
    st.tables[1, :10] = st.tables[0, :10]
    st.tables[2] = st.tables[0, 3]  # one block four times over
    st.dev[0] = torch.from_numpy(st.tables).cuda()
    st.check(st.run())


def test_lengths_beyond_the_bounds_are_left_out():
    """A sequence longer than max_seq_len, or with more queries than keys, writes
    nothing; its neighbours are right (to the bound: the step's lengths decide where
    its keys are cut)."""
    st = Step(14, [100, 50, 300], [1, 2, 1], 8, 2, 64, junk=False)
    want = st.run()
    st.dev[1].copy_(torch.tensor([100, 1, 300], dtype=torch.int32))
    got = st.run()
    assert torch.isnan(got[1:3]).all()
    st.check(torch.cat([got[:1], want[1:3], got[3:]]))
    st.dev[1].copy_(torch.tensor([301, 50, 300], dtype=torch.int32))
    got = st.run()
    assert torch.isnan(got[0]).all()
    st.check(torch.cat([want[:1], got[1:]]))


def test_no_sequence_has_work():
    st = Step(15, [16, 0], [0, 0], 8, 2, 64, junk=False, extra_tokens=3)
    out = torch.full_like(st.q, 2.0)
    st.run(out=out)
    assert (out == 2.0).all()


def test_many_sequences():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 60, 1300)
    st = Step(11, lens, (lens > 0) * rng.integers(0, 2, 1300), 4, 2, 64, junk=False)
    st.check(st.run())


@pytest.mark.parametrize("spread,q_spread", [(30.0, 4.0), (1e-4, 1e-4), (1.0, 1e20), (1.0, 1e-30)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_scores(spread, q_spread, dtype):
    """Peaked rows, flat rows, and queries far from 1 (with a scale that undoes it)."""
    st = Step(5, [700, 90, 1000], [1, 70, 2], 8, 2, 128, dtype, spread, q_spread)
    if q_spread > 100 or q_spread < 1e-10:
        st.scale = st.scale / q_spread
    st.check(st.run())


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 30.0])
def test_vanishing_and_large_scales(scale):
    st = Step(6, [700, 90, 100] + [300] * 14, [1, 70, 2] + [200] * 14, 32, 8, 64, q_spread=1e-3)
    st.scale = scale
    st.check(st.run())


def test_rows_behind_the_last_sequence_stay():
    st = Step(8, [50, 200, 33], [1, 100, 2], 8, 2, 64, extra_tokens=9)
    out = torch.full_like(st.q, 5.0)
    st.run(out=out)
    st.check(out)
    assert (out[int(st.qsl[-1]):] == 5.0).all()


def test_stream_and_graph_follow_the_device_lengths():
    st = Step(9, [600, 1500, 40], [1, 1, 1], 8, 2, 128, junk=False)
    want = st.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = st.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, got)
    out = torch.empty_like(st.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run(out=out)
    g.replay()
    assert torch.equal(out, want)
    st.lens = np.array([77, 900, 33], np.int32)
    st.dev[1].copy_(torch.from_numpy(st.lens))
    g.replay()
    st.check(out)


def test_append_then_attend_as_a_decode_loop():
    """Prompt chunk and decodes: rotate and append, then attend, step by step; the
    queries that the append rotated, the rows that it stored."""
    from tests.test_rope_append_gpu import table
    hq, hkv, d, steps = 8, 2, 64, 4
    rng = np.random.default_rng(21)
    cs_host = table(2000, d)
    cs = torch.from_numpy(cs_host).cuda()
    lens = np.array([37, 0, 200], np.int32)
    blocks = 60
    tables = rng.permutation(blocks).reshape(3, 20).astype(np.int32)
    cache = lib.new_fp4_cache(blocks, hkv, d)
    rows = {s: [] for s in range(3)}  # (codes and scales) of each stored token
    ws = lib.new_fp4_workspace(3, 400, hq, hkv, d)
    for step in range(steps + 1):
        ql = lens + np.array([0, 90, 0], np.int32) if step == 0 else np.ones(3, np.int32)
        before = np.zeros(3, np.int32) if step == 0 else lens
        lens = before + ql
        t = int(ql.sum())
        pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, ql)])
        seq = np.repeat(np.arange(3), ql)
        slots = tables[seq, pos // 16] * 16 + pos % 16
        qkv = torch.from_numpy(rng.standard_normal((t, hq + 2 * hkv, d)).astype(np.float32))
        q, k, v = qkv.bfloat16().cuda().split([hq, hkv, hkv], 1)
        q_rot = lib.rope_append_fp4(q, k, v, cache, torch.from_numpy(slots).long().cuda(),
                                    torch.from_numpy(pos).long().cuda(), cs, k_scale=0.5)
        qsl = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
        out = torch.empty_like(q_rot)
        lib.attention_varlen_fp4(out, q_rot, cache, *(torch.from_numpy(x).cuda() for x in
                                                      (tables, lens, qsl)),
                                 max_query_len=int(ql.max()), max_seq_len=320, scale=d ** -0.5,
                                 workspace=ws, k_scale=0.5)
        kc, ks = fp4_side.quantise(fp4_side.rotate_f32(k.float().cpu().numpy(), cs_host, pos,
                                                       False), 0.5)
        vc, vs = fp4_side.quantise(v.float().cpu().numpy(), 1.0)
        pool = cache.cpu().numpy()
        for i in range(t):
            rows[seq[i]].append((kc[i], ks[i], vc[i], vs[i]))
        want_pool = np.zeros_like(pool)
        for s in range(3):
            for p_, r in enumerate(rows[s]):
                for h in range(hkv):
                    fp4_side.put_row(want_pool[tables[s, p_ // 16], h], p_ % 16, d, r[0][h],
                                     r[1][h], r[2][h], r[3][h])
        assert np.array_equal(pool, want_pool)
        st = Step.__new__(Step)
        st.qsl, st.q64, st.pool, st.tables, st.lens = qsl, q_rot.double().cpu().numpy(), pool, tables, lens
        st.scale, st.k_scale, st.v_scale, st.dtype, st.ws = d ** -0.5, 0.5, 1.0, "bf16", ws
        st.check(out)


def test_binding_refusals():
    st = Step(1, [20], [1], 8, 2, 64)
    with pytest.raises(TypeError):
        lib.attention_varlen_fp4(st.q, st.q, st.cache, st.dev[0].long(), *st.dev[1:],
                                 max_query_len=1, max_seq_len=20, scale=1.0, workspace=st.ws)
    with pytest.raises(ValueError):
        st.run(seq_lens_host=np.array([1, 2], np.int32), query_start_loc_host=st.qsl)
    for bad in (dict(scale=0.0), dict(k_scale=-1.0), dict(v_scale=float("inf")),
                dict(max_seq_len=1000), dict(max_query_len=30), dict(workspace=st.ws[:512]),
                dict(seq_lens_host=np.array([21], np.int32), query_start_loc_host=st.qsl)):
        with pytest.raises(lib.PAError):
            st.run(**bad)
    with pytest.raises(lib.PAError):
        st.run(out=st.q)
    keep = st.q
    for q in (keep.cpu(), keep[:, :4], keep[..., ::2]):
        st.q = q
        with pytest.raises(ValueError):
            st.run(out=torch.empty_like(keep))
    st.q = keep
    with pytest.raises(TypeError):
        st.run(out=torch.empty_like(keep, dtype=torch.float32))
    st.cache = st.cache[..., :1000].contiguous()
    with pytest.raises(TypeError):
        st.run()


def test_mixed_step_side_by_side_is_joined_to_the_stream():
    """Decodes and chunks with host copies may run on two streams: work queued after the
    call sees every row, and a second call on the workspace starts after it."""
    qls = [1] * 40 + [200] * 10
    lens = [900 + 37 * i for i in range(40)] + [200 + 51 * i for i in range(10)]
    st = Step(77, lens, qls, 32, 8, 128, junk=False)
    want = st.run()
    st.check(want)
    out = torch.empty_like(st.q)
    copies = []
    for _ in range(3):
        out.fill_(float("nan"))
        st.run(host=True, out=out)
        copies.append(out.clone())
    st.check(copies[0])
    assert torch.equal(copies[0], copies[1]) and torch.equal(copies[0], copies[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run(host=True, out=out)
    out.fill_(float("nan"))
    g.replay()
    assert torch.equal(out, copies[0])
