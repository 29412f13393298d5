"""The paged 8-bit key/value cache and its attention in plain numpy, 64 bits.

A cache is a dict: k, v (uint8 codes), k_scale, v_scale of one layer, in the
documented layouts (k [pages][heads][block][dim], v [pages][heads][block/16]
[dim][16]).  A batch is (table, kv_len, row_off), numpy int32.
"""
from __future__ import annotations

import numpy as np

EXP_MIN, EXP_MAX = -64, 119


def code_values() -> np.ndarray:
    """The 256 e4m3 values: (-1)^s 2^(e-7) (1 + m/8), subnormal at e = 0, NaN at e = 15, m = 7."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e > 0, (8.0 + m) * np.exp2(e - 10.0), m * 2.0 ** -9)
    mag = np.where((e == 15) & (m == 7), np.nan, mag)
    return np.where(c >> 7 == 1, -mag, mag)


_POS = code_values()[:127]


def to_code(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code, ties to the even one; beyond 448 saturates; non-finite is NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0.0), 448.0)
    hi = np.searchsorted(_POS, a)  # first code >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(np.isfinite(x), c, 127)
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def scale_exp(amax: float) -> int:
    if amax == 0:
        return EXP_MIN
    e = int(np.ceil(np.log2(amax / 448.0)))
    while amax > 448.0 * 2.0 ** e:
        e += 1
    while amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return min(max(e, EXP_MIN), EXP_MAX)


def _v_slot(cache, page, t):
    """[heads][dim] view of token t of a page's values."""
    return cache["v"][page, :, t // 16, :, t % 16]


def rows_of(batch):
    """(sequence, row, position) of every row."""
    table, kv_len, row_off = batch
    for i in range(len(kv_len)):
        m = int(row_off[i + 1] - row_off[i])
        for j in range(m):
            yield i, int(row_off[i]) + j, int(kv_len[i]) - m + j


def page_of(cache, batch, i, pos):
    block = cache["k"].shape[2]
    table = batch[0]
    p = pos // block
    if pos < 0 or p >= table.shape[1]:
        return -1
    page = int(table[i, p])
    return page if 0 <= page < cache["k"].shape[0] else -1


def append(cache, new_k, new_v, batch) -> None:
    """new_k, new_v: float64 [rows][heads][dim]; changes the cache in place."""
    lut = code_values()
    block, heads = cache["k"].shape[2], cache["k"].shape[1]
    groups = {}
    for i, r, pos in rows_of(batch):
        page = page_of(cache, batch, i, pos)
        if page >= 0:
            groups.setdefault((i, pos // block, page), []).append((r, pos % block))
    for (_, _, page), rows in groups.items():
        t0 = rows[0][1]
        for name, x in (("k", new_k), ("v", new_v)):
            slot = (lambda t: cache["k"][page, :, t]) if name == "k" else (lambda t: _v_slot(cache, page, t))
            for h in range(heads):
                val = np.abs(np.stack([x[r, h] for r, _ in rows]))
                val = val[np.isfinite(val)]
                e = scale_exp(float(val.max()) if val.size else 0.0)
                if t0 > 0:
                    old = int(np.round(np.log2(cache[name + "_scale"][page, h])))
                    e = max(e, old)
                    if e > old:
                        for t in range(t0):
                            slot(t)[h] = to_code(lut[slot(t)[h]] * 2.0 ** (old - e))
                for r, t in rows:
                    slot(t)[h] = to_code(x[r, h] * 2.0 ** -e)
                cache[name + "_scale"][page, h] = 2.0 ** e


def read(cache, batch):
    """Rows of the cache, float64 (k, v), [rows][heads][dim]; NaN where there is no page."""
    lut = code_values()
    n, (heads, dim) = int(batch[2][-1]), (cache["k"].shape[1], cache["k"].shape[3])
    k, v = np.full((n, heads, dim), np.nan), np.full((n, heads, dim), np.nan)
    block = cache["k"].shape[2]
    for i, r, pos in rows_of(batch):
        page = page_of(cache, batch, i, pos)
        if page < 0:
            continue
        k[r] = lut[cache["k"][page, :, pos % block]] * cache["k_scale"][page].astype(np.float64)[:, None]
        v[r] = lut[_v_slot(cache, page, pos % block)] * cache["v_scale"][page].astype(np.float64)[:, None]
    return k, v


def attention(cache, q, batch, causal=True, window=0, scale=None):
    """q float64 [rows][query heads][dim].  Returns (out, bound): bound is the
    largest error that the stated roundings allow in each output: the
    probabilities and the output in bf16 (2^-8 relative each), scores, the
    exponential and the sums in fp32."""
    block, heads, dim = cache["k"].shape[2], cache["k"].shape[1], cache["k"].shape[3]
    hq = q.shape[1]
    scale = dim ** -0.5 if scale is None else scale
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    table, kv_len, row_off = batch
    u8, u24 = 2.0 ** -8, 2.0 ** -24
    for i in range(len(kv_len)):
        n, r0, r1 = int(kv_len[i]), int(row_off[i]), int(row_off[i + 1])
        m = r1 - r0
        if m == 0 or n <= 0:
            continue
        hist = (table[i:i + 1], np.array([n]), np.array([0, n]))
        k, v = read(cache, hist)
        for j in range(m):
            hi = n - m + j + 1 if causal else n
            lo = max(0, hi - window) if causal and window else 0
            if hi <= lo:
                continue
            for h in range(hq):
                kk, vv = k[lo:hi, h * heads // hq], v[lo:hi, h * heads // hq]
                s = (kk @ q[r0 + j, h]) * scale
                mag = (np.abs(kk) @ np.abs(q[r0 + j, h])) * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ vv
                # a score's error: its products' sum and its own scaling, in the exponent
                ds = u24 * ((dim + 4) * mag + 4 * np.abs(s) + 4 * np.abs(s).max())
                rel = np.exp(ds) * (1 + 8 * u24) - 1
                dp = p * rel + p * rel.dot(p)  # in the numerator and through the sum
                total = (hi - lo + 64) * u24   # sums over the tokens, in any order
                out[r0 + j, h] = o
                err = dp @ np.abs(vv) + (p @ np.abs(vv)) * (u8 * (1 + rel.max()) + 2 * total)
                bound[r0 + j, h] = err + u8 * (np.abs(o) + err)
    return out, bound
