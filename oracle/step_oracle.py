"""4-bit weights, the norms and rotation of queries and keys, and sampling, in
plain numpy, 64 bits.

4-bit weights are (codes uint8 [dout][din/2], scales uint8 [dout][din/32]); a
batch is (kv_len, row_off), numpy int32.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def q4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 [dout][din]; groups whose scale byte is not in 2 .. 252 are NaN."""
    dout, half = codes.shape
    c = np.empty((dout, 2 * half), np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    b = scales.astype(int)
    s = np.where((b >= 2) & (b <= 252), np.exp2(b - 127.0), np.nan)
    return v * np.repeat(s, GROUP, 1)


def q4_quantize(w: np.ndarray):
    """codes and scales of float64 weights [dout][din]."""
    dout, din = w.shape
    g = w.reshape(dout, din // GROUP, GROUP)
    codes = np.zeros(g.shape, np.uint8)
    scales = np.zeros(g.shape[:2], np.uint8)
    for i in range(dout):
        for j in range(din // GROUP):
            x = g[i, j]
            if not np.isfinite(x).all():
                scales[i, j] = 255
                continue
            e = -125
            while e < 125 and np.abs(x).max() > 6 * 2.0 ** e:
                e += 1
            scales[i, j] = e + 127
            a = np.minimum(np.abs(x) / 2.0 ** e, 6.0)
            d = np.abs(a[:, None] - LEVELS[None, :])
            near = d == d.min(1, keepdims=True)  # two of them halfway: the even code
            code = np.array([min(np.flatnonzero(n), key=lambda k: k % 2) for n in near], np.uint8)
            codes[i, j] = code | (np.signbit(x) << 3)
    codes = codes.reshape(dout, din)
    return codes[:, 0::2] | codes[:, 1::2] << 4, scales


def positions(batch, n_rows: int):
    """(row, position) of every row that a sequence has."""
    kv_len, row_off = batch
    for i in range(len(kv_len)):
        m = int(row_off[i + 1]) - int(row_off[i])
        for j in range(m):
            yield int(row_off[i]) + j, int(kv_len[i]) - m + j


def qk_norm_rotary(x, weight, eps, batch, freqs, interleaved=False, factor=1.0):
    """x [n][heads][dim] -> (result, bound on the error of one fp32 pass whose
    result is rounded to bf16 once); rows without a sequence are NaN."""
    n, _, dim = x.shape
    rot = 2 * len(freqs)
    out, bound = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    u = 2.0 ** -24
    for r, pos in positions(batch, n):
        y = x[r].copy()
        rel = 0.0
        if weight is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
            # dim + 1 sums (halved by the root), mean, root, division, two products: half a step each
            rel = (dim / 2 + 6) * u
        err = np.abs(y) * rel
        angle = pos * np.asarray(freqs)
        c, s = np.cos(angle), np.sin(angle)
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ya, yb, ea, eb = y[:, a], y[:, b], err[:, a], err[:, b]
        # sin and cos: the angle's rounding (pi/4 u), the series' (2 u) and its
        # end (2.5e-9, under u), the factor's (u), and 64-bit angles of far positions
        es = 5 * u + np.abs(angle) * 2.0 ** -51
        y[:, a] = factor * (ya * c - yb * s)
        y[:, b] = factor * (ya * s + yb * c)
        # two products and a sum: three half steps at most on either product
        both = abs(factor) * ((np.abs(ya) + np.abs(yb)) * (es + 3 * u) + (ea + eb) * 1.01)
        err[:, a] = err[:, b] = both
        out[r], bound[r] = y, err * 1.01 + (np.abs(y) + err) * 2.0 ** -8 + 2.0 ** -134
    return out, bound


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0) -> int:
    """The token of one row (logits float64)."""
    x = np.where(np.isnan(logits), -np.inf, logits)
    top = x.max()
    if top == -np.inf:
        return -1
    if not temperature > 0:
        return int(np.flatnonzero(x == top)[0])
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / temperature))
    w = np.where(x == -np.inf, 0.0, np.where(np.isnan(w), 0.0, w))
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    w = w[order]
    cum = np.cumsum(w)
    kept = len(x)
    if top_k > 0:
        kept = min(kept, top_k)
    if top_p < 1:
        reached = np.flatnonzero(cum >= top_p * cum[kept - 1])
        kept = min(kept, int(reached[0]) + 1)
    if min_p > 0:
        kept = min(kept, max(1, int((w >= min(min_p, 1.0)).sum())))
    aim = min(max(u, 0.0), 1 - 2.0 ** -24) * cum[kept - 1]
    at = np.flatnonzero(cum[:kept] > aim)
    return int(order[at[0] if len(at) else kept - 1])


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None) -> np.ndarray:
    get = lambda a, i, off: off if a is None else a[i].item()
    return np.array([sample_row(logits[i], float(u[i]), get(temperature, i, 1.0), get(top_k, i, 0), get(top_p, i, 1.0),
                                get(min_p, i, 0.0)) for i in range(len(logits))], np.int32)
