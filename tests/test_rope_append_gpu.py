"""pa_rope_append, pa_rope_append_fp4 and pa_gather_fp4 against numpy.

Every value is a fixed sequence of fp32 operations, each rounded once, so the
bits are compared; the fp32 formula itself is within its roundings of the fp64
one (a CPU test)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_469_b200 import lib
from paged_kv_cache_469_b200.inputs import f32_to_bf16_bits
from tests import fp4_side


def table(longest, r):
    a = np.arange(longest)[:, None] * 10000.0 ** (-np.arange(0, r, 2) / max(r, 1))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_fp32_rotation_is_the_formula(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 3, 64)).astype(np.float32)
    pos = rng.integers(0, 4000, 50)
    cs = table(4000, 48)
    got = fp4_side.rotate_f32(x, cs, pos, interleaved).astype(np.float64)
    want = x.astype(np.float64)
    for j in range(24):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + 24)
        c, s = cs[pos, j].astype(np.float64)[:, None], cs[pos, j + 24].astype(np.float64)[:, None]
        want[..., a], want[..., b] = (x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s)
    # two products and a sum, half a step each
    bound = 2.0 ** -24 * (2 * np.abs(x).max(-1, keepdims=True) * 2 + np.abs(want))
    assert (np.abs(got - want) <= bound).all()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def make(seed, tokens, hq, hkv, d, dtype, fused):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((tokens, hq + 2 * hkv, d)).astype(np.float32)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    dev = torch.from_numpy(x).to(dt).cuda()
    parts = dev.split([hq, hkv, hkv], dim=1)
    q, k, v = parts if fused else [p.contiguous() for p in parts]
    values = dev.float().cpu().numpy()
    return rng, q, k, v, values[:, :hq], values[:, hq:hq + hkv], values[:, hq + hkv:]


def rounded(x, dtype):
    return x.astype(np.float32) if dtype == "f32" else f32_to_bf16_bits(x)


CASES = [(1, 32, 8, 128, "bf16", 128, False, True), (1, 1, 1, 64, "f32", 64, False, False),
         (37, 8, 2, 64, "bf16", 64, False, True), (37, 8, 2, 64, "bf16", 32, True, True),
         (130, 4, 4, 128, "f32", 96, False, True), (130, 5, 1, 128, "bf16", 64, True, False),
         (700, 32, 8, 128, "bf16", 128, False, True), (2500, 3, 1, 64, "f32", 0, False, False),
         (2500, 32, 4, 64, "bf16", 64, False, False), (64, 0, 2, 128, "bf16", 128, False, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hq,hkv,d,dtype,r,interleaved,fused",
                         CASES + [(33, 6, 2, 128, "bf16", 48, False, True),
                                  (33, 6, 2, 64, "f32", 16, False, True)])
def test_rope_append_bits(tokens, hq, hkv, d, dtype, r, interleaved, fused):
    rng, q, k, v, qv, kv, vv = make(tokens + d, tokens, hq, hkv, d, dtype, fused)
    blocks = tokens // 16 + 5
    slots = rng.permutation(blocks * 16)[:tokens]
    slots[rng.random(tokens) < 0.1] = rng.choice([-1, -16, blocks * 16, 1 << 40])
    longest = 5000
    pos = rng.integers(0, longest, tokens)
    pos[rng.random(tokens) < 0.05] = rng.choice([-1, longest, -(1 << 40)])
    cs = table(longest, r)
    seen = (pos >= 0) & (pos < longest) if r else np.ones(tokens, bool)
    near = np.where(seen, pos, 0)
    caches = [torch.randn(blocks, hkv, 16, d, device="cuda").to(k.dtype) for _ in range(2)]
    want = [c.view(torch.int16 if dtype == "bf16" else torch.float32).cpu().numpy().copy()
            for c in caches]
    if dtype == "bf16":
        want = [w.view(np.uint16) for w in want]
    q_out = torch.full((tokens, hq, d), 7.0, dtype=k.dtype, device="cuda")
    lib.rope_append(q, k, v, *caches, torch.from_numpy(slots).cuda(),
                    torch.from_numpy(pos).cuda() if r else None,
                    torch.from_numpy(cs).cuda() if r else None, q_out=q_out,
                    interleaved=interleaved)
    rot = (lambda x: fp4_side.rotate_f32(x, cs, near, interleaved)) if r else (lambda x: x)
    wq = np.where(seen[:, None, None], rot(qv), np.float32(7))
    assert np.array_equal(bits(q_out), rounded(wq, dtype).view(np.uint8))
    new_k, new_v = rounded(rot(kv), dtype), rounded(vv, dtype)
    for i in range(tokens):
        if seen[i] and 0 <= slots[i] < blocks * 16:
            want[0][slots[i] // 16, :, slots[i] % 16] = new_k[i]
            want[1][slots[i] // 16, :, slots[i] % 16] = new_v[i]
    for c, w in zip(caches, want):
        assert np.array_equal(bits(c), w.view(np.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hq,hkv,d,dtype,r,interleaved,fused",
                         CASES + [(33, 6, 2, 128, "bf16", 48, True, True)])
def test_rope_append_fp4_bytes_and_gather(tokens, hq, hkv, d, dtype, r, interleaved, fused):
    rng, q, k, v, qv, kv, vv = make(tokens + d + 1, tokens, hq, hkv, d, dtype, fused)
    blocks = tokens // 16 + 5
    slots = rng.permutation(blocks * 16)[:tokens]
    slots[rng.random(tokens) < 0.1] = -1
    longest = 5000
    pos = rng.integers(0, longest, tokens)
    cs = table(longest, r)
    k_scale, v_scale = 0.37, 1.0
    before = rng.integers(0, 256, (blocks, hkv, 18 * d), dtype=np.uint8)
    before[..., 16 * d:] &= 0x7e  # scales: finite, positive
    cache = torch.from_numpy(before).cuda()
    q_out = lib.rope_append_fp4(q, k, v, cache, torch.from_numpy(slots).cuda(),
                                torch.from_numpy(pos).cuda() if r else None,
                                torch.from_numpy(cs).cuda() if r else None, k_scale=k_scale,
                                v_scale=v_scale, interleaved=interleaved)
    rot = (lambda x: fp4_side.rotate_f32(x, cs, pos, interleaved)) if r else (lambda x: x)
    assert np.array_equal(bits(q_out), rounded(rot(qv), dtype).view(np.uint8))
    want = before.copy()
    kc, ks = fp4_side.quantise(rot(kv), k_scale)
    vc, vs = fp4_side.quantise(vv, v_scale)
    for i in range(tokens):
        if slots[i] >= 0:
            for h in range(hkv):
                fp4_side.put_row(want[slots[i] // 16, h], slots[i] % 16, d, kc[i, h], ks[i, h],
                                 vc[i, h], vs[i, h])
    assert np.array_equal(cache.cpu().numpy(), want)

    # rows back as values, of any slots, in any order; others left as they are
    read = rng.integers(0, blocks * 16, 45)
    read[3], read[40] = -1, blocks * 16
    for out_type in (torch.float32, torch.bfloat16):
        ko = torch.full((45, hkv, d), 3.0, dtype=out_type, device="cuda")
        vo = torch.full((45, hkv, d), 3.0, dtype=out_type, device="cuda")
        lib.gather_fp4(cache, torch.from_numpy(read).cuda(), k_scale=k_scale, v_scale=v_scale,
                       k_out=ko, v_out=vo)
        values = fp4_side.tile_values(want, d)
        for got, x, g in zip((ko, vo), values, (k_scale, v_scale)):
            rows = np.float32(3) * np.ones((45, hkv, d), np.float32)
            for i, sl in enumerate(read):
                if 0 <= sl < blocks * 16:
                    rows[i] = x[sl // 16, :, sl % 16].astype(np.float32) * np.float32(g)
            exact = rounded(rows, "f32" if out_type == torch.float32 else "bf16")
            assert np.array_equal(bits(got), exact.view(np.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("g", [1.0, 0.37, 3.3e-4, 2.0 ** -61, 1.7e-30, 2.0 ** 59, 4.1e25])
def test_quantiser_next_to_its_ties(g):
    """Values on both sides of every border between two codes, one and two units of the
    last place off it, under every scale and tensor scales of any size."""
    rng = np.random.default_rng(int(abs(np.log2(g)) * 7))
    tokens, d, g = 1000, 128, np.float32(g)
    scale = fp4_side.E4M3[rng.integers(8, 126, (tokens, d // 16))].astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        unit = (scale * g)[..., None]
        ties = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5], np.float32)
        x = ties[rng.integers(0, 7, (tokens, d // 16, 16))] * unit
        for _ in range(2):
            off = rng.integers(-1, 2, x.shape)
            x = np.where(off == 0, x, np.nextafter(x, np.float32(np.inf) * off, dtype=np.float32))
        x[..., 3:4] = 6 * unit
    x = (x * rng.choice(np.array([-1, 1], np.float32), x.shape)).reshape(tokens, 1, d)
    assert np.isfinite(x).all()
    rows, cache = torch.from_numpy(x).cuda(), lib.new_fp4_cache(63, 1, d)
    lib.rope_append_fp4(rows[:, :0], rows, rows, cache, torch.arange(tokens, device="cuda"), None,
                        None, k_scale=float(g), v_scale=float(g))
    want = np.zeros((63, 1, 18 * d), np.uint8)
    c, s = fp4_side.quantise(x, g)
    for i in range(tokens):
        fp4_side.put_row(want[i // 16, 0], i % 16, d, c[i, 0], s[i, 0], c[i, 0], s[i, 0])
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.gpu
def test_quantiser_at_its_borders():
    """Exact ties, values at and past the largest, zeros, subnormal scales, infinities
    and NaN."""
    d = 64
    rows = np.zeros((9, 1, d), np.float32)
    ties = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, -.25, -.75, -1.25, -1.75, -2.5, -3.5,
                     -5, -6], np.float32)
    for i, s in enumerate([1, 1.125, 2.0 ** -6 * 1.75, 448, 2.0 ** -9]):
        rows[i, 0, :16] = ties * np.float32(s)
        rows[i, 0, 16:32] = ties * np.float32(s) * np.float32(1 + 2.0 ** -20)
    rows[5, 0, :] = 1e6
    rows[6, 0, ::7] = 1e-30
    rows[7, 0, 5] = np.inf
    rows[7, 0, 20] = -np.inf
    rows[8, 0, 9] = np.nan
    x = torch.from_numpy(rows).cuda()
    cache = lib.new_fp4_cache(1, 1, d)
    slots = torch.arange(9, device="cuda")
    lib.rope_append_fp4(x[:, :0], x, x, cache, slots, None, None)
    want = np.zeros((1, 1, 18 * d), np.uint8)
    c, s = fp4_side.quantise(rows, 1.0)
    for i in range(9):
        fp4_side.put_row(want[0, 0], i, d, c[i, 0], s[i, 0], c[i, 0], s[i, 0])
    got = cache.cpu().numpy()
    assert np.array_equal(got[..., 16 * d:], want[..., 16 * d:])
    kg, _ = lib.gather_fp4(cache, slots, dtype=torch.float32)
    kw = fp4_side.tile_values(want, d)[0][0, 0, :9].astype(np.float32)
    # the codes of a NaN group mean nothing: its values are NaN whatever they are
    assert np.array_equal(kg[:, 0].cpu().numpy(), kw, equal_nan=True)
    assert np.isnan(kw[8, :16]).all() and np.isfinite(kw[8, 16:]).all()


@pytest.mark.gpu
def test_in_place_stream_and_graph():
    rng, q, k, v, qv, kv, vv = make(5, 21, 8, 2, 128, "bf16", False)
    cs = torch.from_numpy(table(600, 128)).cuda()
    pos = torch.from_numpy(rng.integers(0, 600, 21)).cuda()
    slots = torch.from_numpy(rng.permutation(64)[:21]).cuda()
    kc, vc = (torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want = lib.rope_append(q, k, v, kc, vc, slots, pos, cs)
    k2, v2, q2 = torch.zeros_like(kc), torch.zeros_like(vc), q.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lib.rope_append(q2, k, v, k2, v2, slots, pos, cs, q_out=q2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q2, want) and torch.equal(k2, kc) and torch.equal(v2, vc)
    # captured: a replay reads what the tensors hold then
    q3 = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.rope_append(q, k, v, k2, v2, slots, pos, cs, q_out=q3)
    pos.copy_((pos + 7) % 600)
    want = lib.rope_append(q, k, v, kc, vc, slots, pos, cs)
    k2.zero_()
    g.replay()
    assert torch.equal(q3, want) and torch.equal(k2[kc != 0], kc[kc != 0])


@pytest.mark.gpu
def test_binding_refusals():
    q, k = (torch.zeros(3, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    cs = torch.zeros(10, 64, device="cuda")
    ok = dict(q=q, k=k, v=k, k_cache=kc, v_cache=kc.clone(), slot_mapping=slots, positions=slots,
              cos_sin=cs)
    for bad, err in ((dict(slot_mapping=slots.int()), TypeError),
                     (dict(positions=slots.int()), TypeError),
                     (dict(positions=None), TypeError),
                     (dict(positions=slots[:2]), ValueError),
                     (dict(slot_mapping=slots[:2]), ValueError),
                     (dict(cos_sin=cs.double()), TypeError),
                     (dict(cos_sin=cs[:, ::2]), ValueError),
                     (dict(q=q.float()), TypeError),
                     (dict(k_cache=kc.float()), TypeError),
                     (dict(k_cache=kc[:, :1]), ValueError),
                     (dict(v=k.transpose(0, 1)), ValueError),
                     (dict(k=k.cpu()), ValueError),
                     (dict(cos_sin=torch.zeros(10, 40, device="cuda")), lib.PAError),
                     (dict(q_out=k.new_empty(3, 4, 64)[..., :32]), ValueError)):
        with pytest.raises(err):
            lib.rope_append(**{**ok, **bad})
    with pytest.raises(lib.PAError):  # overlapping, not in place
        buf = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
        lib.rope_append(**{**ok, "q": buf[:3], "q_out": buf[1:]})
    cache = lib.new_fp4_cache(2, 2, 64)
    with pytest.raises(lib.PAError):
        lib.rope_append_fp4(q, k, k, cache, slots, slots, cs, k_scale=0.0)
    with pytest.raises(TypeError):
        lib.rope_append_fp4(q, k, k, cache.float(), slots, slots, cs)
    with pytest.raises(ValueError):
        lib.gather_fp4(cache, slots, k_out=k.new_empty(2, 2, 64))
