"""Inputs, wanted results and error bars of the 4-bit pools, on the host."""
import numpy as np

import oracle
from rope_cases import Append, values
from span_cases import Decode


def shifted(x, nbytes):
    """A copy of tensor x that begins nbytes behind a multiple of 256 bytes."""
    raw = x.new_empty(x.numel() + (nbytes + 256) // x.element_size())
    skip = (-raw.data_ptr() % 256 + nbytes) // x.element_size()
    y = raw[skip:skip + x.numel()].view(x.shape).copy_(x)
    assert y.data_ptr() % 256 == nbytes and y.is_contiguous()
    return y


def pool(r, nb, hkv, bs):
    """Random rows of different sizes, as they are stored."""
    x = r.standard_normal((nb, hkv, bs, 128)) * 2.0 ** r.integers(-6, 7, (nb, hkv, bs, 1))
    x[..., ::16] *= 4
    return oracle.pack_rows(x.astype(np.float32))


class Append4(Append):
    def __init__(self, seed, tokens, hq, hkv, rot, bs, nb, **kw):
        super().__init__(seed, "bf16", tokens, hq, hkv, 128, rot, bs, nb, **kw)
        r = np.random.default_rng(seed + 1000)
        self.k_cache, self.v_cache = pool(r, nb, hkv, bs), pool(r, nb, hkv, bs)

    def want(self):
        """The pools behind the call (the stated float32 arithmetic)."""
        kc, vc = self.k_cache.copy(), self.v_cache.copy()
        k, v = self.rotated32(self.k), values(self.v)
        for t, s in enumerate(self.written()):
            if s >= 0:
                kc[s // self.bs, :, s % self.bs] = oracle.pack_rows(k[t])
                vc[s // self.bs, :, s % self.bs] = oracle.pack_rows(v[t])
        return kc, vc


class Decode4(Decode):
    """span_cases.Decode over 4-bit pools: rows that nobody sees have NaN scales."""

    def __init__(self, seed, lens, q_len, hq, hkv, bs, window=0, sinks=0, spread=0, **kw):
        super().__init__(seed, "bf16", lens, q_len, hq, hkv, 128, bs, window, sinks, **kw)
        r = np.random.default_rng(seed + 1000)
        pools = []
        for c in (self.k_cache, self.v_cache):
            x = values(c)
            unseen = np.isnan(x).any(-1)
            x = np.where(unseen[..., None], np.float32(1), x)
            x = x * (np.float32(2.0) ** r.integers(-spread, spread + 1, x.shape[:3] + (1,)).astype(np.float32))
            rows = oracle.pack_rows(x)
            rows[unseen] = r.integers(0, 256, (int(unseen.sum()), 72))
            rows[unseen, 64:] = 0xFF
            pools.append(rows)
        self.k_cache, self.v_cache = pools
        self.dtype = "fp4"

    def want(self):
        k, v = (oracle.unpack_rows(c) for c in (self.k_cache, self.v_cache))
        return oracle.decode_window_f64(values(self.q).astype(np.float64), k, v, self.tables, self.lens, self.scale,
                                        self.window, self.sinks)

    def bar(self, out, parts):
        """As for e4m3 pools: the weights are halves, 2^-11 of each and 2^-35 of the largest
        (subnormal steps of 2^-25 under the factor 2^10); q's elements 2^-32 of the largest."""
        d = self.q.shape[-1]
        rel = 2 * 2.0 ** -22 * d * parts["dots"][..., None] + 2.0 ** -20
        qmax = np.abs(values(self.q)).max(-1, keepdims=True).astype(np.float64)
        dq = self.scale * 2.0 ** -32 * qmax * parts["ksum"][..., None]
        vmax = np.nanmax(np.abs(np.where(np.isfinite(v := oracle.unpack_rows(self.v_cache)), v, 0)))
        tiny = 2.0 ** -34 * vmax * float(self.lens.max())
        return 2.0 ** -8 * np.abs(out) + (2.0 ** -11 * 1.01 + rel + 2 * dq) * parts["mag"] + tiny + 1e-37
