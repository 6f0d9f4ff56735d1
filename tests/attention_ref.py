"""Definitions of the attention beside the indexer in plain numpy, in double precision where they are
computed numbers, and bounds on what a kernel's rounding may add.  Shares no code with the package."""
import math

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every e4m3 number by its byte (127 is NaN)
E4M3 = np.array([(b & 7) / 8 * 2.0 ** -6 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(127)])


def nearest_even(x, grid):
    """Index of the grid value nearest to each x >= 0, ties to the even index, the last one above the grid."""
    hi = np.clip(np.searchsorted(grid, x), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    a, b = x - grid[lo], grid[hi] - x
    return np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def pack(x, g):
    """Rows x [..., d] (fp32) -> (code bytes [..., d/2], scale bytes [..., d/16]), the divisions in fp32."""
    d = x.shape[-1]
    x = np.where(np.isnan(x), np.float32(0), x.astype(np.float32)).reshape(*x.shape[:-1], d // 16, 16)
    g = np.float32(g)
    with np.errstate(all="ignore"):
        raw = np.abs(x).max(-1) / (g * np.float32(6))
        s8 = nearest_even(np.minimum(raw.astype(np.float64), 448.0), E4M3)
        unit = (E4M3[s8].astype(np.float32) * g)[..., None]
        y = np.where(unit > 0, x / np.where(unit > 0, unit, np.float32(1)), np.float32(0))
    code = nearest_even(np.minimum(np.abs(y).astype(np.float64), 6.0), LEVELS) + 8 * (np.signbit(y) & (unit > 0))
    code = code.astype(np.uint8).reshape(*x.shape[:-2], d)
    out = np.zeros((*x.shape[:-2], d // 2), np.uint8)
    for e in range(d):
        out[..., byte_of(e, d)] |= code[..., e] << (4 * (e % 2))
    return out, s8.astype(np.uint8)


def byte_of(e, d):
    return (d // 8) * (e % 16 // 4) + 2 * (e // 16) + e % 4 // 2


def unpack(codes, scales):
    """(code bytes, scale bytes) -> values in double."""
    d = codes.shape[-1] * 2
    e = np.arange(d)
    nib = (codes[..., byte_of(e, d)] >> (4 * (e % 2)).astype(np.uint8)) & 15
    v = LEVELS[nib & 7] * np.where(nib >= 8, -1.0, 1.0)
    return v * E4M3[scales][..., e // 16]


def views(pool, page, d):
    """Code rows [pages, H_kv, 2, page, d/2] and scale rows [.., d/16] of a numpy pool."""
    n, h = pool.shape[:2]
    a, b = pool[..., :page * d // 2], pool[..., page * d // 2:]
    return a.reshape(n, h, 2, page, d // 2), b.reshape(n, h, 2, page, d // 16)


def cache_rows(pool, table_row, pos, page, d):
    """K, V [len(pos), H_kv, d] (double) of the logical positions of one sequence."""
    codes, scales = views(pool, page, d)
    pg, at = table_row[pos // page], pos % page
    x = unpack(codes[pg, :, :, at], scales[pg, :, :, at])
    return x[:, :, 0], x[:, :, 1]


def attend(q, k, v, scale, seen=None):
    """q [m, Hq, d], k, v [l, Hkv, d] -> out, lse, weights [Hq, m, l]; seen [m, l] bool; double."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    G = q.shape[1] // k.shape[1]
    kk, vv = np.repeat(k, G, axis=1), np.repeat(v, G, axis=1)
    s = np.einsum("mhd,lhd->hml", q, kk) * scale
    if seen is not None:
        s = np.where(seen[None], s, -np.inf)
    top = s.max(-1, initial=-np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    p = np.exp(s - safe[..., None])
    total = p.sum(-1)
    with np.errstate(divide="ignore"):
        lse = safe + np.log(total)
    p = p / np.where(total > 0, total, 1.0)[..., None]
    return np.einsum("hml,lhd->mhd", p, vv), lse.T, p


def attend_tolerance(q, k, v, scale, p, dtype, weight_eps, weight_floor=0.0):
    """Per-output bound [m, Hq, d] for outputs of `dtype` ("bf16" or "f32"), and the bound of a logit.

    A logit is a sum of d products in fp32 (at most 2^-23 of the sum of magnitudes for each of the d
    additions); an error of e in every logit moves each weight by at most 2 e of itself (its own and the
    sum's), the exponential and the sum add 2^-20, and rounding a weight adds weight_eps of it (1.06 times
    that: the next bound's slack); the output is then rounded to its type (half a step).
    weight_floor: absolute error of a weight below the normal range of the type it is rounded to."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    G = q.shape[1] // k.shape[1]
    kk, vv = np.repeat(k, G, axis=1), np.repeat(v, G, axis=1)
    mag = np.einsum("mhd,lhd->hml", np.abs(q), np.abs(kk)) * scale
    e = q.shape[-1] * 2.0 ** -23 * (mag.max() if mag.size else 0.0) + 2.0 ** -22
    pv = np.einsum("hml,lhd->mhd", p, np.abs(vv))
    out = np.abs(np.einsum("hml,lhd->mhd", p, vv))
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    # sums over tokens in fp32: 2^-24 a step, at most one step a token
    run = 2.0 ** -24 * max(16, k.shape[0])
    return out * step + pv * (2 * e + 2.0 ** -20 + 1.06 * weight_eps + run) * (1 + step) + weight_floor * np.abs(vv).sum(0)[None] + 1e-30, e


def evict(acc, n, keep, sink, recent):
    """Tokens that stay of one sequence, ascending."""
    if n <= keep:
        return list(range(n))
    key = [(-math.inf if math.isnan(a) else a) for a in acc[:n].tolist()]
    nan = [math.isnan(a) for a in acc[:n].tolist()]
    mid = sorted(range(sink, n - recent), key=lambda s: (nan[s], -key[s], s))[:keep - sink - recent]
    return sorted(list(range(sink)) + mid + list(range(n - recent, n)))
