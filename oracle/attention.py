"""FP64 oracle of the attention calls (numpy): head norms with the position
rotation, the 8-bit paged cache, attention over it, from their definitions. No
code of the CUDA path; the cache is walked token by token."""
from __future__ import annotations

import numpy as np

BLOCK = 16
# the 127 magnitudes of e4m3 by code; code 127 is NaN
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])
E4M3[127] = np.nan


def decode(codes):
    codes = np.asarray(codes).astype(np.int64)
    return np.where(codes >= 128, -1.0, 1.0) * E4M3[codes & 127]


def encode(x):
    """Nearest e4m3 code by distance, a tie to the even code, NaN for what is not
    finite. |x| <= 448."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x)
    a = np.abs(np.where(fine, x, 0.0))
    up = np.searchsorted(E4M3[:127], a)                  # the first magnitude >= a
    up = np.minimum(up, 126)
    down = np.maximum(up - 1, 0)
    hi, lo = E4M3[up] - a, a - E4M3[down]
    code = np.where((hi < lo) | ((hi == lo) & (up % 2 == 0)), up, down)
    code = np.where(E4M3[up] == a, up, code)
    return np.where(fine, code + 128 * np.signbit(x), 127).astype(np.uint8)


def exponent(values):
    """The smallest e >= -120 with max|finite| <= 448 * 2^e."""
    v = np.abs(values[np.isfinite(values)])
    top = v.max() if v.size else 0.0
    e = -120
    while top > 448 * 2.0 ** e:
        e += 1
    return e


def scale_of(byte):
    return np.nan if byte == 255 else 2.0 ** (int(byte) - 127)


def norm_rope(x, w, cos_sin, pos, eps, interleaved=False, plus_one=False):
    """x [T][heads][D] float64 -> the same, unrounded."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * (w + (1.0 if plus_one else 0.0))
    if cos_sin is None:
        return y
    half = cos_sin.shape[1] // 2
    out = y.copy()
    for t, p in enumerate(pos):
        if not 0 <= p < len(cos_sin):
            out[t] = np.nan
            continue
        c, s = cos_sin[p, :half], cos_sin[p, half:]
        i = np.arange(half) * (2 if interleaved else 1)
        j = i + (1 if interleaved else half)
        out[t][:, i] = y[t][:, i] * c - y[t][:, j] * s
        out[t][:, j] = y[t][:, j] * c + y[t][:, i] * s
    return out


def place(table, page, j):
    return table[j // page], j % page


def append(codes, scales, rows, table, first, side):
    """Tokens `rows` [n][heads][D] (values as they are quantised) of one sequence
    from position `first` on, into side `side` of codes and scales."""
    page = codes.shape[3]
    n = len(rows)
    last = first + n
    for start in range(max(first, 0) // BLOCK * BLOCK, last, BLOCK):
        pg, at = place(table, page, start)
        mine = range(max(start, first, 0), min(start + BLOCK, last))
        for h in range(codes.shape[2]):
            new = np.array([rows[j - first][h] for j in mine])
            byte = exponent(new) + 127
            was = int(scales[pg, side, h, at // BLOCK])
            older = range(start, min(start + BLOCK, max(first, 0)))
            if len(older):
                byte = max(byte, was)
                if byte > was:
                    for j in older:
                        v = decode(codes[pg, side, h, j % page]) * 2.0 ** (was - byte)
                        codes[pg, side, h, j % page] = encode(v)
            scales[pg, side, h, at // BLOCK] = byte
            for j in mine:
                codes[pg, side, h, j % page] = encode(rows[j - first][h] * 2.0 ** (127 - byte))


def held(codes, scales, table, n):
    """Keys and values [2][n][heads][D] of a sequence's first n tokens."""
    page = codes.shape[3]
    out = np.empty((2, n, codes.shape[2], codes.shape[4]))
    for j in range(n):
        pg, at = place(table, page, j)
        if not 0 <= pg < len(codes):
            out[:, j] = np.nan
            continue
        s = scales[pg, :, :, at // BLOCK].astype(np.int64)
        s = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
        out[:, j] = decode(codes[pg, :, :, at]) * s[..., None]
    return out


def attention(q, k, v, scale, absent=None):
    """One sequence: q [n][hq][D] its last n rows, k and v [kv][hkv][D]; absent
    [kv] marks tokens that are not there. Returns (out [n][hq][D], weights times
    |v|, largest sum of |products|) with 0 where a row sees nothing."""
    n, hq, _ = q.shape
    kv, hkv, D = k.shape
    out, size = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    big = np.zeros((n, hq, 1))
    there = np.ones(kv, dtype=bool) if absent is None else ~absent
    with np.errstate(invalid="ignore"):
        for i in range(n):
            see = there & (np.arange(kv) <= kv - n + i)
            if not see.any():
                continue
            for h in range(hq):
                g = h // (hq // hkv)
                kk, vv = k[see, g], v[see, g]
                t = kk @ q[i, h] * scale
                p = np.exp(t - np.max(t))
                p = p / p.sum()
                out[i, h] = p @ vv
                size[i, h] = p @ np.abs(vv)
                big[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, size, big
