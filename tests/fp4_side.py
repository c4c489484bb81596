"""The rotating append and the 4-bit cache in numpy, for the tests: every element
at its own place, in loops or whole-array arithmetic, sharing nothing with the
library.  fp32 where the definition is (each operation rounded once), fp64 else."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
_b = np.arange(127)
E4M3 = np.where(_b < 8, _b * 2.0 ** -9, (8 + _b % 8) * 2.0 ** (_b // 8 - 10.0))  # bytes 0 .. 126


def e4m3_value(byte):
    """fp64 value of scale bytes (127: NaN; the sign bit is never set by the library)."""
    byte = np.asarray(byte)
    return np.where(byte == 127, np.nan, E4M3[np.minimum(byte, 126)])


def _nearest_even(x, grid):
    """Index of the nearest grid value, ties to the even index, past the end the last."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def rotate_f32(x, cos_sin, positions, interleaved):
    """fp32 rotation of [T, H, D] rows, each product and sum rounded on its own."""
    x = np.asarray(x, np.float32)
    r = cos_sin.shape[1]
    c, s = cos_sin[positions][:, None, :r // 2], cos_sin[positions][:, None, r // 2:]
    i1 = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    i2 = i1 + 1 if interleaved else i1 + r // 2
    y = x.copy()
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def quantise(x, g):
    """(codes [.., D], scale bytes [.., D / 16]) of fp32 rows under the tensor scale g."""
    x = np.asarray(x, np.float32)
    grp = x.reshape(*x.shape[:-1], -1, 16)
    with np.errstate(invalid="ignore", over="ignore"):
        raw = np.abs(grp).max(-1) / np.float32(6 * np.float32(g))
    nan = np.isnan(raw)
    byte = np.where(nan, 127, _nearest_even(np.where(nan, 0, raw).astype(np.float64), E4M3))
    s = e4m3_value(byte).astype(np.float32)
    with np.errstate(invalid="ignore"):
        d = np.where(s > 0, s * np.float32(g), np.float32(np.inf)).astype(np.float32)
        y = grp / d[..., None]
    code = _nearest_even(np.abs(np.nan_to_num(y, nan=0.0)).astype(np.float64), E2M1[:8])
    code = code + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def put_row(tile, off, d, k_codes, k_scales, v_codes, v_scales):
    """One token's codes and scales into its tile, byte by byte."""
    for dim in range(0, d, 2):
        tile[off * (d // 2) + dim // 2] = k_codes[dim] | k_codes[dim + 1] << 4
        c, within = dim // (d // 8), dim % (d // 8)
        h, t, i = off // 2 % 2, off // 4, off % 2
        tile[8 * d + (((h * 8 + c) * 4 + t) * 2 + i) * (d // 16) + within // 2] = \
            v_codes[dim] | v_codes[dim + 1] << 4
    for grp in range(d // 16):
        tile[16 * d + off * (d // 16) + grp] = k_scales[grp]
        tile[17 * d + grp * 16 + off] = v_scales[grp]


def tile_values(tiles, d):
    """K and V of tiles [..., 18 d]: fp64 [..., 16, d], without the tensor scales."""
    token, dim = np.arange(16)[:, None], np.arange(d)[None]
    kb = token * (d // 2) + dim // 2
    wide = d // 8
    vb = 8 * d + (((token // 2 % 2 * 8 + dim // wide) * 4 + token // 4) * 2 + token % 2) * \
        (wide // 2) + dim % wide // 2
    ks, vs = 16 * d + token * (d // 16) + dim // 16, 17 * d + dim // 16 * 16 + token
    out = []
    for at, sc in ((kb, ks), (vb, vs)):
        code = tiles[..., at] >> (4 * (dim % 2)) & 15
        out.append(E2M1[code] * e4m3_value(tiles[..., sc]))
    return out


def random_tiles(rng, n, d, spread=1.0):
    """n tiles of normal K and V rows, quantised."""
    kc, ks = quantise(rng.standard_normal((n, 16, d)).astype(np.float32) * spread, 1.0)
    vc, vs = quantise(rng.standard_normal((n, 16, d)).astype(np.float32), 1.0)
    kb = kc[..., 0::2] | kc[..., 1::2] << 4
    vb = (vc[..., 0::2] | vc[..., 1::2] << 4).reshape(n, 4, 2, 2, 8, d // 16)
    return np.concatenate([kb.reshape(n, -1), vb.transpose(0, 2, 4, 1, 3, 5).reshape(n, -1),
                           ks.reshape(n, -1), vs.transpose(0, 2, 1).reshape(n, -1)], 1)


def attention(q, kv_cache, tables, seq_lens, qsl, scale, k_scale, v_scale):
    """fp64 outputs, and per output what the error bound needs: sum_k p |v|, and the
    row's largest scale * sum_d |q k|."""
    hq, d = q.shape[1:]
    hkv = kv_cache.shape[1]
    out = np.zeros(q.shape)
    mass = np.zeros(q.shape)
    reach = np.zeros(q.shape[:2])
    for s, n in enumerate(seq_lens):
        ql = qsl[s + 1] - qsl[s]
        if ql == 0:
            continue
        tiles = kv_cache[tables[s, :-(-n // 16)]]
        k, v = tile_values(tiles, d)
        k = k.transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n] * float(np.float32(k_scale))
        v = v.transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n] * float(np.float32(v_scale))
        for h in range(hq):
            kh, vh = k[h * hkv // hq], v[h * hkv // hq]
            rows = q[qsl[s]:qsl[s + 1], h]
            x = rows @ kh.T * scale
            future = np.arange(n)[None] > (n - ql + np.arange(ql))[:, None]
            x[future] = -np.inf
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[qsl[s]:qsl[s + 1], h] = p @ vh
            mass[qsl[s]:qsl[s + 1], h] = p @ np.abs(vh)
            reach[qsl[s]:qsl[s + 1], h] = (np.abs(rows) @ np.abs(kh).T * scale).max(-1)
    return out, mass, reach
