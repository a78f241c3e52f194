"""Causal attention of packed prompts in 64 bits, sequence by sequence."""
from __future__ import annotations

import numpy as np


def prefill_f64(q, k_pool, v_pool, tables, lens, starts, scale, window=0, sinks=0):
    """q [T, Hq, D]; pools [NB, Hkv, bs, D] in float64; sequence b's new tokens are rows
    starts[b] .. starts[b + 1] - 1 and the last of its lens[b] tokens.  Returns the output
    (rows of no sequence: NaN) and what its error bars are made of: sum p |V| and the largest
    scale * sum |q| |k| over the seen tokens."""
    T, Hq, D = q.shape
    Hkv, bs = k_pool.shape[1:3]
    group = Hq // Hkv
    out, mag, dots = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros(q.shape[:2])
    for b in range(len(lens)):
        r0, r1, L = int(starts[b]), int(starts[b + 1]), int(lens[b])
        if r1 <= r0:
            continue
        out[r0:r1] = 0
        p = L - (r1 - r0) + np.arange(r1 - r0)[:, None]
        t = np.arange(max(L, 0))
        see = (t <= p) & ((p - t < window) | (t < sinks) if window > 0 else True)
        t = np.flatnonzero(see.any(0))
        if len(t) == 0:
            continue
        see = see[:, t]
        some = see.any(1)
        page = tables[b][t // bs]
        for h in range(Hkv):
            k, v = k_pool[page, h, t % bs], v_pool[page, h, t % bs]
            for i in range(h * group, (h + 1) * group):
                s = np.where(see, scale * (q[r0:r1, i] @ k.T), -np.inf)
                w = np.exp(s - np.where(some, s.max(1), 0.0)[:, None])
                w /= np.where(some, w.sum(1), 1.0)[:, None]
                out[r0:r1, i] = w @ v
                mag[r0:r1, i] = w @ np.abs(v)
                dots[r0:r1, i] = np.where(see, scale * (np.abs(q[r0:r1, i]) @ np.abs(k).T), 0).max(1)
    return out, dict(mag=mag, dots=dots)
