"""Inputs and wanted results of the rotating appends, on the host."""
import numpy as np

import oracle
import pa_inputs


def table(max_position, rot, base=10000.0):
    half = rot // 2
    angle = np.arange(max_position)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def values(a):
    """Storage (float32 or bf16 bits) -> float32 values."""
    return oracle.widen(a, "bf16").astype(np.float32) if a.dtype == np.uint16 else a


def storage(a, dtype):
    return pa_inputs.to_storage(np.asarray(a, np.float32), dtype)


class Append:
    """Rows of q, k, v as slices of one matrix, with slots, positions and pools."""

    def __init__(self, seed, dtype, tokens, hq, hkv, d, rot, bs, nb, max_position=64,
                 interleaved=False, slots=None, positions=None):
        r = np.random.default_rng(seed)
        self.dtype, self.hq, self.hkv, self.d, self.bs, self.nb = dtype, hq, hkv, d, bs, nb
        self.interleaved = interleaved
        bf = "f32" if dtype == "f32" else "bf16"
        self.qkv = storage(r.standard_normal((tokens, (hq + 2 * hkv) * d)), bf)
        x = self.qkv.reshape(tokens, -1, d)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        self.cos_sin = table(max_position, rot)
        self.positions = (r.integers(0, max_position, tokens) if positions is None
                          else np.asarray(positions)).astype(np.int64)
        self.slots = (r.permutation(nb * bs)[:tokens] if slots is None
                      else np.asarray(slots)).astype(np.int64)
        shape = (nb, hkv, bs, d)
        if dtype in ("f32", "bf16"):
            self.k_cache = storage(r.standard_normal(shape), dtype)
            self.v_cache = storage(r.standard_normal(shape), dtype)
        else:
            self.k_cache, self.k_scales = self._pool8(r, shape)
            self.v_cache, self.v_scales = self._pool8(r, shape)
            self.k_scale = r.uniform(0.01, 0.03, hkv).astype(np.float32)
            self.v_scale = r.uniform(0.01, 0.03, hkv).astype(np.float32)

    @staticmethod
    def _pool8(r, shape):
        x = (r.standard_normal(shape) * 2.0 ** r.integers(-3, 3, shape[:2] + (1, 1))).astype(np.float32)
        s = np.array([[oracle.power_of_two_scale(np.abs(x[p, h]).max()) for h in range(shape[1])]
                      for p in range(shape[0])], np.float32)
        return oracle.e4m3_encode(x / s[:, :, None, None]), s

    def live(self):
        return (self.positions >= 0) & (self.positions < len(self.cos_sin))

    def rows(self):
        return self.cos_sin[np.where(self.live(), self.positions, 0)]

    def rotated32(self, x):
        return oracle.rotate_f32(values(x), self.rows(), self.interleaved)

    def rotated64(self, x):
        return oracle.rotate_f64(values(x).astype(np.float64), self.rows(), self.interleaved)

    def written(self):
        """Slot of each token, -1 where nothing is written."""
        ok = self.live() & (self.slots < self.nb * self.bs)
        return np.where(ok, self.slots, -1)


def kept_in_pages(slots, bs, behind=48):
    """Which tokens a page-scaled append writes, of those with a slot (>= 0): a page's tokens
    one after another but for unwritten ones, no more than the page's size, none more than
    `behind` behind the first, none of a page that another page's tokens have interrupted."""
    kept, begun = np.zeros(len(slots), bool), set()
    page = start = count = None
    for t, s in enumerate(slots):
        if s < 0:
            continue
        if s // bs != page:
            page, start, count, fresh = s // bs, t, 0, s // bs not in begun
            begun.add(page)
        if fresh and t - start <= behind and count < bs:
            kept[t] = True
            count += 1
    return kept
