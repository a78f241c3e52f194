"""Windowed decode with sinks in 64 bits, sequence by sequence and row by row."""
from __future__ import annotations

import numpy as np


def seen(length, q_len, j, window, sinks):
    """Positions that new token j of q_len attends to, increasing."""
    p = length - q_len + j
    t = np.arange(max(0, p + 1))
    return t if window <= 0 else t[(p - t < window) | (t < sinks)]


def decode_window_f64(q, k_pool, v_pool, tables, lens, scale, window=0, sinks=0, v_scales=None):
    """q [B, q_len, Hq, D]; pools [NB, Hkv, bs, D] in float64 (dequantised).  Returns the
    output and what its error bars are made of: sum p |V|, the largest
    scale * sum |q| |k| over the seen tokens, the largest sum |k|, and (v_scales given)
    max(p vs) * sum |V / vs|."""
    B, q_len, Hq, D = q.shape
    Hkv, bs = k_pool.shape[1:3]
    group = Hq // Hkv
    out = np.zeros(q.shape)
    mag, dots, ksum, wmax = np.zeros(q.shape), np.zeros(q.shape[:3]), np.zeros(q.shape[:3]), np.zeros(q.shape)
    for b in range(B):
        for j in range(q_len):
            t = seen(int(lens[b]), q_len, j, window, sinks)
            if len(t) == 0:
                continue
            page = tables[b][t // bs]
            for h in range(Hkv):
                k, v = k_pool[page, h, t % bs], v_pool[page, h, t % bs]
                for i in range(h * group, (h + 1) * group):
                    s = scale * (k @ q[b, j, i])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[b, j, i] = w @ v
                    mag[b, j, i] = w @ np.abs(v)
                    dots[b, j, i] = scale * (np.abs(k) @ np.abs(q[b, j, i])).max()
                    ksum[b, j, i] = np.abs(k).sum(1).max()
                    if v_scales is not None:
                        vs = v_scales[page, h]
                        wmax[b, j, i] = (w * vs).max() * np.abs(v / vs[:, None]).sum(0)
    return out, dict(mag=mag, dots=dots, ksum=ksum, wmax=wmax)
