"""Rows of 4-bit pools, in plain numpy: 64 bytes of e2m1 codes and 8 scales for 128 columns.

Tables of all values and the nearest one by distance; nothing is computed from bit fields
but the tables' own entries.
"""
from __future__ import annotations

import numpy as np

# code -> value: sign, two exponent bits (bias 1), one fraction bit
E2M1_VALUES = np.array([(-1.0) ** (c >> 3) * (0.5 * (c & 1) if (c >> 1) & 3 == 0 else
                                             2.0 ** (((c >> 1) & 3) - 1) * (1 + 0.5 * (c & 1))) for c in range(16)])


def scale_value(byte) -> float:
    """A scale byte: five exponent bits (bias 15), three fraction bits, no sign."""
    e, f = byte >> 3, byte & 7
    if e == 31:
        return float("nan") if f else float("inf")
    return f * 2.0 ** -17 if e == 0 else (8 + f) * 2.0 ** (e - 18)


SCALE_VALUES = np.array([scale_value(b) for b in range(256)])
MOST = int(np.searchsorted(SCALE_VALUES[:248], 10240.0))
NAN_SCALE = 0xFF


def _nearest(values, x):
    """Index of the nearest of increasing `values` to each x >= 0, ties to the even index."""
    i = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    below, above = x - values[i - 1], values[i] - x
    down = (below < above) | ((below == above) & (i % 2 == 1))
    return np.where(x >= values[-1], len(values) - 1, np.where(down, i - 1, i))


def pack_rows(x):
    """float32 rows [..., 128] as uint8 rows [..., 72]."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], 8, 16)
    nan = np.isnan(b).any(-1)
    mag = np.where(np.isnan(b), np.float32(0), np.abs(b))
    y = mag.max(-1) / np.float32(6)
    scale = _nearest(SCALE_VALUES[:MOST + 1], y.astype(np.float64)).astype(np.uint8)
    s = SCALE_VALUES[scale].astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(s > 0, mag / s, np.float32(0))
    code = _nearest(E2M1_VALUES[:8], z.astype(np.float64)).astype(np.uint8) | (((b < 0) & (s > 0)) * 8).astype(np.uint8)
    code = code.reshape(*x.shape[:-1], 64, 2)
    return np.concatenate([code[..., 0] | code[..., 1] << 4, np.where(nan, NAN_SCALE, scale).astype(np.uint8)], -1)


def unpack_rows(rows):
    """uint8 rows [..., 72] as float64 values [..., 128]."""
    codes = np.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).reshape(*rows.shape[:-1], 8, 16)
    return (E2M1_VALUES[codes] * SCALE_VALUES[rows[..., 64:]][..., None]).reshape(*rows.shape[:-1], 128)
