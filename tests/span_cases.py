"""Inputs, wanted results and error bars of the windowed / page-scaled decodes, on the host."""
import numpy as np

import oracle
import pa_inputs
from rope_cases import storage, values


class Decode:
    """Pools that hold only what some new token sees: every other slot is NaN, and table
    entries of pages that nobody sees are not pages at all."""

    def __init__(self, seed, dtype, lens, q_len, hq, hkv, d, bs, window=0, sinks=0, spread=0, std=1.0,
                 first_norm=1.0):
        r = np.random.default_rng(seed)
        self.dtype, self.q_len, self.hkv, self.bs, self.window, self.sinks = dtype, q_len, hkv, bs, window, sinks
        self.lens = np.asarray(lens, np.int32)
        self.scale = float(np.float32(d ** -0.5))
        B, width = len(lens), max(1, -(-max(lens) // bs)) + 1
        seen = [sorted({int(t) for j in range(q_len) for t in oracle.seen(L, q_len, j, window, sinks)}) for L in lens]
        pages = [sorted({t // bs for t in s}) for s in seen]
        self.nb = sum(map(len, pages)) + 3
        order = r.permutation(self.nb)
        self.tables = r.choice([-1, -7, self.nb, 2 ** 31 - 1], (B, width)).astype(np.int32)
        at = 0
        mask = np.zeros((self.nb, bs), bool)
        for b in range(B):
            self.tables[b, pages[b]] = order[at:at + len(pages[b])]
            at += len(pages[b])
            t = np.asarray(seen[b], int)
            mask[self.tables[b][t // bs], t % bs] = True
        shape = (self.nb, hkv, bs, d)
        bf = "f32" if dtype == "f32" else "bf16"
        self.q = storage(r.standard_normal((B, q_len, hq, d)) * std, bf)
        pools, self.scales = [], []
        for n in range(2):
            x = (r.standard_normal(shape) * std).astype(np.float32)
            if n and first_norm != 1.0:                       # first pages' V of another size
                x[self.tables[:, 0][self.tables[:, 0] < self.nb]] *= first_norm
            if dtype == "fp8":
                x *= np.float32(2.0) ** r.integers(-spread, spread + 1, shape[:2] + (1, 1)).astype(np.float32)
                amax = np.abs(x).max((2, 3))
                s = np.array([[oracle.power_of_two_scale(a) for a in row] for row in amax], np.float32)
                s *= np.where(r.random(s.shape) < 0.5, np.float32(1.0), np.float32(1.25))   # any positive scale will do
                c = oracle.e4m3_encode(x / s[:, :, None, None])
                c = np.where(mask[:, None, :, None], c, np.uint8(0x7F)).astype(np.uint8)
                self.scales.append(s)
                pools.append(c)
            else:
                x = np.where(mask[:, None, :, None], x, np.float32(np.nan))
                pools.append(storage(x, bf))
        self.k_cache, self.v_cache = pools

    def want(self):
        if self.dtype == "fp8":
            k, v = (oracle.E4M3_VALUES[c] * s[:, :, None, None].astype(np.float64)
                    for c, s in zip((self.k_cache, self.v_cache), self.scales))
        else:
            k, v = (values(c).astype(np.float64) for c in (self.k_cache, self.v_cache))
        vs = self.scales[1].astype(np.float64) if self.dtype == "fp8" else None
        return oracle.decode_window_f64(values(self.q).astype(np.float64), k, v, self.tables, self.lens, self.scale,
                                        self.window, self.sinks, vs)

    def bar(self, out, parts):
        """Largest error of each output.  Scores: D products and sums in float32, 2^-22 D of
        the sum of their magnitudes (sums may be cut instead of rounded), so a weight is
        within 2 ds + 2^-20 of itself (exp2's approximation).  bf16: half a step of 2^-8 for
        each weight and for the result.  e4m3: q's elements become halves, scaled so that the
        row's largest is at least 2^7: exact but for 2^-25 (subnormal steps), 2^-32 of the
        largest; the weights are halves too, 2^-11 of each and 2^-35 of the largest."""
        d = self.q.shape[-1]
        ds = 2.0 ** -22 * d * parts["dots"][..., None]
        rel = 2 * ds + 2.0 ** -20
        if self.dtype == "f32":
            return rel * parts["mag"] + 1e-37
        bar = 2.0 ** -8 * np.abs(out) + 1e-37
        if self.dtype == "bf16":
            return bar + (2.0 ** -8 * 1.01 + rel) * parts["mag"]
        qmax = np.abs(values(self.q)).max(-1, keepdims=True).astype(np.float64)
        dq = self.scale * 2.0 ** -32 * qmax * parts["ksum"][..., None]
        return bar + (2.0 ** -11 * 1.01 + rel + 2 * dq) * parts["mag"] + 2.0 ** -34 * parts["wmax"]
