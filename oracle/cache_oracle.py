"""fp64 oracle of the cache-side operators (test infrastructure only): rotary
positions with several axes, the quantised paged cache, attention over a shared
prefix. Written from the definitions in include/tsel.h; shares no code with the
library."""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(base, sections, layout):
    """(radians per position step, axis) per pair; layout "sectioned",
    "interleaved" or "per_axis"."""
    pairs, n = sum(sections), len(sections)
    if layout == "interleaved":
        axis = [i % n if i // n < sections[i % n] else 0 for i in range(pairs)]
    else:
        axis = [a for a, s in enumerate(sections) for _ in range(s)]
    if layout == "per_axis":
        freq = [base ** (-j / s) for s in sections for j in range(s)]
    else:
        freq = [base ** (-i / pairs) for i in range(pairs)]
    return np.asarray(freq, np.float64), np.asarray(axis, np.int64)


def rope(x, pos, freq, axis, adjacent=False, inverse=False):
    """x [T, H, d] (any real type) rotated by pos [T, axes]; fp64."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    n = len(freq)
    # the angle in extended precision: positions reach 2^31
    ang = np.asarray(pos, np.longdouble)[:, axis] * np.asarray(freq, np.longdouble)
    c = np.cos(ang).astype(np.float64)[:, None]
    s = np.sin(ang).astype(np.float64)[:, None] * (-1 if inverse else 1)
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = a * s + b * c
    return y


def _e4m3_values():
    v = np.zeros(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            v[b] = np.nan
        else:
            v[b] = (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) * (-1 if s else 1)
    return v


E4M3 = _e4m3_values()
_GRID = E4M3[:127]   # 0 .. 448


def quantise(x):
    """(codes uint8, exponent bytes uint8) of rows x [..., d]."""
    x = np.asarray(x, np.float64)
    codes = np.zeros(x.shape, np.uint8)
    exps = np.zeros(x.shape[:-1], np.uint8)
    for i in np.ndindex(exps.shape):
        row = x[i]
        if not np.all(np.isfinite(row)):
            exps[i] = 255
            continue
        e = -127
        top = np.max(np.abs(row)) if row.size else 0.0
        while top > 448.0 * 2.0 ** e:
            e += 1
        y = np.abs(row) / 2.0 ** e
        hi = np.clip(np.searchsorted(_GRID, y), 1, 126)
        lo = hi - 1
        up, down = _GRID[hi] - y, y - _GRID[lo]
        c = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
        codes[i] = c | np.where(np.signbit(row), 128, 0)
        exps[i] = e + 127
    return codes, exps


def dequantise(codes, exps):
    e = np.asarray(exps, np.float64)[..., None]
    return np.where(e == 255, np.nan, E4M3[codes] * 2.0 ** (e - 127))


def attention_row(q, k, v, scale):
    """(out [d], lse, abs-weighted mean of v [d], largest sum |q||k| * scale) of
    one query row over keys k, v [n, d]."""
    d = v.shape[1]
    if len(k) == 0:
        return np.zeros(d), -math.inf, np.zeros(d), 0.0
    z = scale * (k @ q)
    m = np.max(z)
    p = np.exp(z - m)
    total = p.sum()
    mag = scale * float(np.max(np.abs(k) @ np.abs(q)))
    return (p @ v) / total, m + math.log(total), (p @ np.abs(v)) / total, mag


def prefix_attention(q, cu, k, v, prefix_rows, suffix_rows, scale):
    """q [T, H, d]; k, v fp64 [slots, Hkv, d] (the cache as values); prefix_rows
    the prefix's slots, suffix_rows[r] those of request r's suffix. Returns (out,
    lse [H, T], abs-weighted v, magnitude of the logits' terms [T, H])."""
    T, H, d = q.shape
    G = H // k.shape[1]
    out, av = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse, mag = np.zeros((H, T)), np.zeros((T, H))
    for r in range(len(cu) - 1):
        n = cu[r + 1] - cu[r]
        for i in range(n):
            t = cu[r] + i
            seen = max(0, min(len(suffix_rows[r]), len(suffix_rows[r]) - n + i + 1))
            rows = np.concatenate([prefix_rows, suffix_rows[r][:seen]]).astype(np.int64)
            for h in range(H):
                out[t, h], lse[h, t], av[t, h], mag[t, h] = attention_row(
                    q[t, h], k[rows, h // G], v[rows, h // G], scale)
    return out, lse, av, mag
