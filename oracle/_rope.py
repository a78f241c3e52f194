"""Rotary positions on the way into the cache, in plain numpy.

``rotate_f64`` is the definition in 64 bits; ``rotate_f32`` is the stated float32
arithmetic (every product and every sum rounded), which decides what an 8-bit code
near a rounding border becomes.  ``page_scale_append`` writes rows into e4m3 pools
with a scale for each page and head, page by page as the call's statement has it.
"""
from __future__ import annotations

import numpy as np

from ._cache_ops import e4m3_encode, e4m3_value

E4M3_VALUES = np.array([e4m3_value(c) for c in range(256)])


def _turn(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    y = x.copy()
    one, two = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
                else (slice(0, rot // 2), slice(rot // 2, rot)))
    a, b = x[..., one], x[..., two]
    y[..., one] = a * cos - b * sin
    y[..., two] = b * cos + a * sin
    return y


def rotate_f64(x, table_rows, interleaved=False):
    """x [T, H, D] (float64), table_rows [T, rot] = cos | sin of each token's position."""
    t = np.asarray(table_rows, np.float64)[:, None, :]
    h = t.shape[-1] // 2
    return _turn(np.asarray(x, np.float64), t[..., :h], t[..., h:], interleaved)


def rotate_f32(x, table_rows, interleaved=False):
    """The same in float32, each operation rounded."""
    t = np.asarray(table_rows, np.float32)[:, None, :]
    h = t.shape[-1] // 2
    return _turn(np.asarray(x, np.float32), t[..., :h], t[..., h:], interleaved)


def power_of_two_scale(amax) -> np.float32:
    """2^k with the least k >= -100 such that amax <= 448 2^k (exact, by comparison)."""
    k = -100
    while float(amax) > 448.0 * 2.0 ** k:
        k += 1
    return np.float32(2.0 ** k)


def page_scale_append(x, slots, codes, scales):
    """Rows x float32 [T, H, D] into codes uint8 [NB, H, bs, D] and scales float32
    [NB, H], in place.  Tokens with a negative slot are left out."""
    bs = codes.shape[2]
    pages = {}
    for t, s in enumerate(slots):
        if s >= 0:
            pages.setdefault(int(s) // bs, []).append((t, int(s) % bs))
    for page, rows in pages.items():
        offs = [o for _, o in rows]
        others = [o for o in range(bs) if o not in offs]
        for h in range(x.shape[1]):
            new = np.stack([x[t, h] for t, _ in rows])
            mag = np.abs(new[np.isfinite(new)])
            need = power_of_two_scale(mag.max() if mag.size else 0.0)
            old = scales[page, h]
            s = need if 0 in offs else max(old, need)
            if 0 not in offs and s > old:
                kept = E4M3_VALUES[codes[page, h, others]].astype(np.float32) * np.float32(old / s)
                codes[page, h, others] = e4m3_encode(kept)
            for t, o in rows:
                codes[page, h, o] = e4m3_encode(x[t, h] / s)
            scales[page, h] = s
