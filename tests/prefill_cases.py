"""Inputs, wanted results and error bars of the prompt attention, on the host."""
import numpy as np

import oracle
from rope_cases import storage, values


class Prompts:
    """Packed prompts over pools that hold only what some new token sees: every other slot is
    NaN, and table entries of pages that nobody sees are not pages at all.  new, had: new and
    earlier tokens of each sequence; before, behind: rows of q of no sequence."""

    def __init__(self, seed, dtype, new, had, hq, hkv, d, bs, window=0, sinks=0, before=0, behind=0, std=1.0):
        r = np.random.default_rng(seed)
        self.dtype, self.hkv, self.bs, self.window, self.sinks = dtype, hkv, bs, window, sinks
        new, had = np.asarray(new), np.asarray(had)
        self.lens = (new + had).astype(np.int32)
        self.starts = (before + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        self.rows = int(self.starts[-1]) + behind
        self.scale = float(np.float32(d ** -0.5))
        B, width = len(new), max(1, -(-int(self.lens.max()) // bs)) + 1
        pages, seen = [], []
        for n, m in zip(new, had):
            p, t = m + np.arange(n)[:, None], np.arange(m + n)
            see = (t <= p) & ((p - t < window) | (t < sinks) if window else True)
            seen.append(np.flatnonzero(see.any(0)))
            pages.append(np.unique(seen[-1] // bs))
        self.nb = sum(map(len, pages)) + 3
        order = r.permutation(self.nb)
        self.tables = r.choice([-1, -7, self.nb, 2 ** 31 - 1], (B, width)).astype(np.int32)
        mask, at = np.zeros((self.nb, bs), bool), 0
        for b in range(B):
            self.tables[b, pages[b]] = order[at:at + len(pages[b])]
            at += len(pages[b])
            mask[self.tables[b][seen[b] // bs], seen[b] % bs] = True
        self.q = storage(r.standard_normal((self.rows, hq, d)) * std, dtype)
        shape = (self.nb, hkv, bs, d)
        self.k_cache, self.v_cache = (
            storage(np.where(mask[:, None, :, None], (r.standard_normal(shape) * std).astype(np.float32), np.float32(np.nan)), dtype)
            for _ in range(2))

    def mine(self):
        """Rows of q that belong to a sequence."""
        m = np.zeros(self.rows, bool)
        m[self.starts[0]:self.starts[-1]] = True
        return m

    def want(self):
        q, k, v = (values(x).astype(np.float64) for x in (self.q, self.k_cache, self.v_cache))
        return oracle.prefill_f64(q, k, v, self.tables, self.lens, self.starts, self.scale, self.window, self.sinks)

    def bar(self, out, parts):
        """Largest error of each output.  Scores: D products and sums in float32, 2^-22 D of
        the sum of their magnitudes (sums may be cut instead of rounded), and the rounding of
        the score times log2(e) to float32 and of its difference from the reference, 2^-22 of
        it; so a weight is within 2 ds + 2^-20 of itself (exp2's approximation).  Sums of n
        weights and of n products: 2 n 2^-24.  bf16: half a step of 2^-8 for each weight and
        for the result."""
        d, n = self.q.shape[-1], int(self.lens.max())
        ds = (2.0 ** -22 * d + 2.0 ** -21) * parts["dots"][..., None]
        rel = 2 * ds + 2.0 ** -20 + 2 * n * 2.0 ** -24
        if self.dtype == "f32":
            return rel * parts["mag"] + 2.0 ** -23 * np.abs(out) + 1e-37
        return 2.0 ** -8 * np.abs(out) + (2.0 ** -8 * 1.01 + rel) * parts["mag"] + 1e-37
