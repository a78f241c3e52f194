"""The rotating appends on the GPU against the oracle.

Bars.  float32: the two products and the sum are each rounded, so a rotated value is
within 2 * 2^-24 (|a cos| + |b sin|) of the 64-bit one, first order; 2^-22 (|a| + |b|)
covers it.  bf16: half a step on top, 2^-8 of the value.  Codes and scales: the
stated float32 arithmetic decides them, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
import rope_cases
from gpu_helpers import DEV, storage_to_host, to_dev

pytestmark = pytest.mark.gpu


class Dev:
    """A rope_cases.Append on the device; q, k, v are slices of one matrix."""

    def __init__(self, c):
        self.c = c
        bf = c.dtype != "f32"
        qkv = to_dev(c.qkv, bf)
        cut = [c.hq * c.d, c.hkv * c.d, c.hkv * c.d]
        self.q, self.k, self.v = (x.unflatten(-1, (-1, c.d)) for x in qkv.split(cut, 1))
        self.kc, self.vc = (to_dev(x, c.dtype == "bf16") for x in (c.k_cache, c.v_cache))
        self.slots, self.pos, self.table = to_dev(c.slots), to_dev(c.positions), to_dev(c.cos_sin)
        self.q_out = torch.full(self.q.shape, -7.0, dtype=self.q.dtype, device=DEV)
        self.errs = torch.zeros(1, dtype=torch.int32, device=DEV)
        if c.dtype == "fp8":
            self.scale = to_dev(c.k_scale), to_dev(c.v_scale)
        if c.dtype == "fp8_block":
            self.scale = to_dev(c.k_scales), to_dev(c.v_scales)

    def call(self, **kw):
        fn = {"fp8": pa.pa_rope_and_cache_fp8, "fp8_block": pa.pa_rope_and_cache_fp8_block}.get(
            self.c.dtype, pa.pa_rope_and_cache)
        args = (self.q_out, self.q, self.k, self.v, self.kc, self.vc, self.slots, self.pos, self.table)
        if self.c.dtype.startswith("fp8"):
            args += self.scale
        fn(*args, interleaved=self.c.interleaved, device_errors=self.errs, **kw)
        return pa.pa_read_device_errors(self.errs)


def _check_rotated(got, c, x, live):
    """Rotated rows of storage x against 64 bits."""
    want = c.rotated64(x)[live]
    mag = np.abs(rope_cases.values(x)).astype(np.float64)[live]
    half = c.cos_sin.shape[1] // 2
    pair = mag.copy()
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c.interleaved
                else (slice(0, half), slice(half, 2 * half)))
    pair[..., one] = pair[..., two] = mag[..., one] + mag[..., two]
    bar = 2.0 ** -22 * pair
    if c.dtype != "f32":
        bar = bar + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(got[live] - want) <= bar)


def _check(c, d):
    """Everything one call wrote, and everything it must leave alone."""
    live, w = c.live(), c.written()
    bf = "f32" if c.dtype == "f32" else "bf16"
    q = rope_cases.values(storage_to_host(d.q_out, bf)).astype(np.float64)
    _check_rotated(q, c, c.q, live)
    assert np.all(q[~live] == -7.0)
    page, off, on = w // c.bs, w % c.bs, w >= 0
    if c.dtype in ("f32", "bf16"):
        gk, gv = storage_to_host(d.kc, c.dtype), storage_to_host(d.vc, c.dtype)
        _check_rotated(np.where(on[:, None, None], rope_cases.values(gk[page, :, off]), 0).astype(np.float64),
                       c, c.k, on)
        kc, vc = c.k_cache.copy(), c.v_cache.copy()
        kc[page[on], :, off[on]] = gk[page[on], :, off[on]]       # checked above
        vc[page[on], :, off[on]] = c.v[on]
        np.testing.assert_array_equal(gk, kc)
        np.testing.assert_array_equal(gv, vc)
        return
    rows = {"k": c.rotated32(c.k), "v": rope_cases.values(c.v)}
    for n, cache, dev, i in (("k", c.k_cache, d.kc, 0), ("v", c.v_cache, d.vc, 1)):
        want = cache.copy()
        if c.dtype == "fp8":
            s = (c.k_scale, c.v_scale)[i]
            want[page[on], :, off[on]] = oracle.e4m3_encode(rows[n][on] / s[None, :, None])
        else:
            s = (c.k_scales, c.v_scales)[i].copy()
            oracle.page_scale_append(rows[n], w, want, s)
            np.testing.assert_array_equal(storage_to_host(d.scale[i], "f32"), s)
        got = storage_to_host(dev, "fp8")
        nan = (want & 0x7F) == 0x7F                               # a NaN's sign is free
        np.testing.assert_array_equal(got[~nan], want[~nan])
        assert np.all((got[nan] & 0x7F) == 0x7F)


def _run_of(spans, bs, seed=0):
    """Slots of sequences in pages of their own, each appending from `had` on; the pages
    are handed out in a shuffled order.  Returns (slots, positions, pages needed)."""
    slots, pos, base = [], [], 0
    pages = sum((had + new - 1) // bs - had // bs + 1 for had, new in spans)
    order = np.random.default_rng(seed).permutation(pages + 3)
    for had, new in spans:
        for p in range(had, had + new):
            slots.append(order[base + p // bs - had // bs] * bs + p % bs)
            pos.append(p)
        base += (had + new - 1) // bs - had // bs + 1
    return slots, pos, pages + 3


@pytest.mark.parametrize("dtype,d,rot", [("f32", 64, 64), ("f32", 128, 48), ("bf16", 64, 16),
                                         ("bf16", 128, 128), ("bf16", 128, 80), ("fp8", 128, 128),
                                         ("fp8", 128, 32)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens,hq,hkv", [(1, 8, 8), (5, 3, 1), (37, 32, 8), (700, 6, 3)])
def test_rotates_and_writes(dtype, d, rot, inter, tokens, hq, hkv):
    bs = 16 if tokens % 2 else 32
    c = rope_cases.Append(tokens + rot, dtype, tokens, hq, hkv, d, rot, bs, tokens // bs + 3,
                          interleaved=inter)
    dv = Dev(c)
    assert dv.call() == 0
    _check(c, dv)


@pytest.mark.parametrize("inter,rot", [(False, 128), (True, 64), (False, 16)])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("spans,hq,hkv", [
    ([(0, 1)], 8, 8), ([(3, 1), (16, 1), (31, 1), (32, 1)], 4, 2), ([(5, 70), (0, 33), (15, 2)], 3, 1),
    ([(0, 900), (31, 500)], 6, 3)])
def test_appends_with_page_scales(spans, hq, hkv, bs, inter, rot):
    slots, pos, nb = _run_of(spans, bs, len(spans))
    c = rope_cases.Append(sum(p for _, p in spans) + bs, "fp8_block", len(slots), hq, hkv, 128, rot, bs,
                          nb, max_position=1024, interleaved=inter, slots=slots, positions=pos)
    dv = Dev(c)
    assert dv.call() == 0
    _check(c, dv)


def test_page_scale_grows_and_earlier_rows_follow():
    """Rows of very different size into one page, one call a row: growing, then not."""
    c = rope_cases.Append(5, "fp8_block", 1, 0, 2, 128, 128, 16, 3, slots=[0], positions=[0])
    kc, ks = c.k_cache, c.k_scales
    vc, vs = c.v_cache, c.v_scales
    first = Dev(c)
    for step, (slot, size) in enumerate([(16, 1e-3), (17, 5.0), (18, 300.0), (19, 1e-4), (20, 7e4), (16, 1.0)]):
        c = rope_cases.Append(50 + step, "fp8_block", 1, 0, 2, 128, 128, 16, 3, slots=[slot], positions=[step])
        c.qkv[:] = rope_cases.storage(rope_cases.values(c.qkv) * np.float32(size), "bf16")
        c.k_cache, c.k_scales, c.v_cache, c.v_scales = kc.copy(), ks.copy(), vc.copy(), vs.copy()
        d = Dev(c)
        d.q = d.q_out = None
        d.kc, d.vc, d.scale = first.kc, first.vc, first.scale
        c.q = c.q[:, :0]
        fn = pa.pa_rope_and_cache_fp8_block
        fn(None, None, d.k, d.v, d.kc, d.vc, d.slots, d.pos, d.table, *d.scale, device_errors=d.errs)
        oracle.page_scale_append(c.rotated32(c.k), c.slots, kc, ks)
        oracle.page_scale_append(rope_cases.values(c.v), c.slots, vc, vs)
        np.testing.assert_array_equal(storage_to_host(d.kc, "fp8"), kc)
        np.testing.assert_array_equal(storage_to_host(d.vc, "fp8"), vc)
        np.testing.assert_array_equal(storage_to_host(d.scale[0], "f32"), ks)
        np.testing.assert_array_equal(storage_to_host(d.scale[1], "f32"), vs)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp8_block"])
def test_padding_uncached_and_bad_tokens(dtype):
    """Negative position: nothing at all.  Negative slot: q alone.  A position past the
    table or a slot past the pool: flagged, and skipped alike."""
    d = 128
    slots = [0, 1, -1, 2, -1, 19, 20, 10 ** 12, 33, -5]
    pos = [0, 1, 2, -1, -1, 3, 64, 4, 63, 7]
    c = rope_cases.Append(9, dtype, 10, 4, 2, d, 128, 16, 4, slots=slots, positions=pos)
    dv = Dev(c)
    assert dv.call() == pa.PA_DEVERR_BAD_SLOT | pa.PA_DEVERR_BAD_POSITION
    _check(c, dv)


def test_special_values_in_page_scaled_rows():
    """Zeros alone, subnormals, infinities, NaN, and the largest finite values."""
    c = rope_cases.Append(11, "fp8_block", 16, 0, 8, 128, 16, 16, 2, slots=range(16, 32),
                          positions=[0] * 16)                     # angle 0: rows as they are
    x = rope_cases.values(c.qkv).reshape(16, -1, 128).copy()
    x[:, 0] = 0.0
    x[:, 1] = 1e-39
    x[3, 2, 5], x[4, 2, 6], x[5, 2, 7] = np.inf, -np.inf, np.nan
    x[:, 3] = 3.3e38
    x[:, 4] = -1e-30
    x[:, 5, 1:] = np.nan
    x[:, 6] = np.inf
    c.qkv[:] = rope_cases.storage(x.reshape(16, -1), "bf16")
    d = Dev(c)
    pa.pa_rope_and_cache_fp8_block(None, None, d.k, d.v, d.kc, d.vc, d.slots, None, None, *d.scale,
                                   device_errors=d.errs)
    assert pa.pa_read_device_errors(d.errs) == 0
    for name, x, cache, s, got, gs in (("k", c.k, c.k_cache, c.k_scales, d.kc, d.scale[0]),
                                       ("v", c.v, c.v_cache, c.v_scales, d.vc, d.scale[1])):
        oracle.page_scale_append(rope_cases.values(x), c.slots, cache, s)
        np.testing.assert_array_equal(storage_to_host(gs, "f32"), s)
        g = storage_to_host(got, "fp8")
        nan = (cache & 0x7F) == 0x7F
        np.testing.assert_array_equal(g[~nan], cache[~nan])
        assert np.all((g[nan] & 0x7F) == 0x7F)


@pytest.mark.parametrize("bs", [16, 32])
def test_more_tokens_than_slots_are_refused(bs):
    slots = [o % bs for o in range(bs + 5)]
    c = rope_cases.Append(12, "fp8_block", bs + 5, 2, 2, 128, 128, bs, 2, slots=slots)
    before = storage_to_host(to_dev(c.k_cache[1:]), "fp8")
    d = Dev(c)
    assert d.call() & pa.PA_DEVERR_BAD_SLOT
    np.testing.assert_array_equal(storage_to_host(d.kc[1:], "fp8"), before)


def test_in_place_and_contiguous_rows():
    c = rope_cases.Append(13, "bf16", 33, 8, 2, 128, 128, 16, 4)
    d = Dev(c)
    d.q, d.k, d.v = d.q.contiguous(), d.k.contiguous(), d.v.contiguous()
    d.q_out = d.q
    assert d.call() == 0
    _check(c, d)


def test_rope_append_equals_the_plain_cache_write_without_rotation():
    c = rope_cases.Append(14, "bf16", 40, 0, 3, 128, 128, 16, 6)
    d = Dev(c)
    pa.pa_rope_and_cache(None, None, d.k, d.v, d.kc, d.vc, d.slots, None, None, device_errors=d.errs)
    kc, vc = to_dev(c.k_cache, True), to_dev(c.v_cache, True)
    pa.pa_reshape_and_cache(d.k.contiguous(), d.v.contiguous(), kc, vc, d.slots, device_errors=d.errs)
    assert torch.equal(d.kc.view(torch.int16), kc.view(torch.int16))
    assert torch.equal(d.vc.view(torch.int16), vc.view(torch.int16))
    assert pa.pa_read_device_errors(d.errs) == 0


def test_slots_past_32_bits_of_elements():
    """A pool of more than 2^32 elements: the last page's rows."""
    hkv, bs, d = 32, 16, 128
    nb = (1 << 32) // (hkv * bs * d) + 5
    kc = torch.zeros(nb, hkv, bs, d, dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    ks, vs = torch.zeros(nb, hkv, device=DEV), torch.zeros(nb, hkv, device=DEV)
    x = torch.ones(2, hkv, d, dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([nb * bs - bs, nb * bs - bs + 1], device=DEV)
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rope_and_cache_fp8_block(None, None, x, x, kc, vc, slots, None, None, ks, vs, device_errors=errs)
    assert pa.pa_read_device_errors(errs) == 0
    assert int((kc[-1] != 0).sum()) == 2 * hkv * d and int((kc[:5] != 0).sum()) == 0
    assert bool((ks[-1] == 2.0 ** -8).all()) and int((ks[:-1] != 0).sum()) == 0


def test_refusals_of_the_python_call():
    c = rope_cases.Append(15, "bf16", 4, 4, 2, 128, 128, 16, 2)
    d = Dev(c)
    ok = dict(q_out=d.q_out, q=d.q, k=d.k, v=d.v, k_cache=d.kc, v_cache=d.vc, slot_mapping=d.slots,
              positions=d.pos, cos_sin=d.table)
    pa.pa_rope_and_cache(**ok)
    for over, kind in ((dict(q=d.q.float()), TypeError), (dict(k=d.k[:3]), ValueError),
                       (dict(v=d.v[..., :64]), ValueError), (dict(k=d.k.transpose(0, 1)), ValueError),
                       (dict(slot_mapping=d.slots.int()), TypeError), (dict(positions=d.pos[:2]), ValueError),
                       (dict(cos_sin=d.table.double()), TypeError), (dict(cos_sin=None), ValueError),
                       (dict(q_out=None), ValueError), (dict(k_cache=d.kc.float()), (TypeError, ValueError)),
                       (dict(cos_sin=d.table[:, :40].contiguous()), pa.PaError),
                       (dict(slot_mapping=d.slots.cpu()), ValueError)):
        with pytest.raises(kind):
            pa.pa_rope_and_cache(**{**ok, **over})


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp8_block"])
def test_prepared_call_given_stream_and_no_tokens(dtype):
    c = rope_cases.Append(16, dtype, 40, 8, 4, 128, 96, 16, 6, slots=list(range(16, 56)))
    d = Dev(c)
    fn = {"fp8": pa.pa_rope_and_cache_fp8, "fp8_block": pa.pa_rope_and_cache_fp8_block}.get(dtype, pa.pa_rope_and_cache)
    scale = d.scale if dtype.startswith("fp8") else ()
    call = fn(d.q_out, d.q, d.k, d.v, d.kc, d.vc, d.slots, d.pos, d.table, *scale, device_errors=d.errs, prepare=True)
    assert isinstance(call, pa.PreparedCall) and bool((d.q_out == -7.0).all())
    call()
    assert pa.pa_read_device_errors(d.errs) == 0
    _check(c, d)
    side = torch.cuda.Stream()
    e = Dev(c)
    side.wait_stream(torch.cuda.current_stream())
    fn(e.q_out, e.q, e.k, e.v, e.kc, e.vc, e.slots, e.pos, e.table, *(e.scale if scale else ()), device_errors=e.errs,
       stream=side)
    side.synchronize()
    _check(c, e)
    before = d.kc.clone()
    fn(d.q_out[:0], d.q[:0], d.k[:0], d.v[:0], d.kc, d.vc, d.slots[:0], d.pos[:0], d.table, *scale)
    assert torch.equal(before.view(torch.uint8), d.kc.view(torch.uint8))


def test_many_decode_tokens_and_mixed_runs():
    """More tokens than one tile's blocks take at once; runs of one token among longer ones,
    runs that begin in one tile and end in the next, padding between sequences."""
    r = np.random.default_rng(17)
    for bs, hkv in ((16, 5), (32, 9)):
        spans = [(int(h), int(n)) for h, n in zip(r.integers(0, 60, 500), np.where(r.random(500) < 0.6, 1, r.integers(1, 50, 500)))]
        slots, pos, nb = _run_of(spans, bs, 3)
        at = np.cumsum([n for _, n in spans])[::7]                 # a padding token after every seventh sequence
        slots, pos = list(np.insert(slots, at, -1)), list(np.insert(pos, at, -1))
        c = rope_cases.Append(18 + bs, "fp8_block", len(slots), 2, hkv, 128, 128, bs, nb, max_position=128,
                              slots=slots, positions=pos)
        d = Dev(c)
        assert d.call() == 0
        _check(c, d)


def test_copy_scales_follows_copied_and_swapped_pages():
    r = torch.Generator(device=DEV).manual_seed(3)
    ks, vs = (torch.rand(7, 3, generator=r, device=DEV) for _ in range(2))
    wk, wv = ks.clone(), vs.clone()
    pairs = torch.tensor([[1, 5], [0, 6], [2, 9], [-1, 3]], device=DEV)
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_copy_scales(ks, vs, ks, vs, pairs, device_errors=errs)
    assert pa.pa_read_device_errors(errs) == pa.PA_DEVERR_BAD_BLOCK
    for s, t in ((1, 5), (0, 6)):
        wk[t], wv[t] = wk[s], wv[s]
    assert torch.equal(ks, wk) and torch.equal(vs, wv)
    hk, hv = torch.zeros(2, 3).pin_memory(), torch.zeros(2, 3).pin_memory()
    pa.pa_copy_scales(ks, vs, hk, hv, torch.tensor([[6, 1], [4, 0]], device=DEV), device_errors=errs)
    assert pa.pa_read_device_errors(errs) == 0
    assert torch.equal(hk, wk[[4, 6]].cpu()) and torch.equal(hv, wv[[4, 6]].cpu())


@pytest.mark.parametrize("spans,hq,hkv,bs", [
    ([(7, 1000)], 5, 5, 16), ([(0, 900), (40, 1200)], 5, 5, 16), ([(0, 3500)], 7, 7, 16), ([(90, 2100)], 12, 3, 32),
    ([(17, 2900), (0, 1333)], 32, 8, 16), ([(3, 9001)], 20, 1, 16), ([(5, 8500)], 36, 2, 32), ([(0, 1700)], 9, 9, 16)])
def test_prompts_of_many_sizes(spans, hq, hkv, bs):
    """From one head of a run at a time to eight, one group of heads or several, q's blocks
    between the runs' blocks or behind them."""
    slots, pos, nb = _run_of(spans, bs, hq)
    c = rope_cases.Append(hq + bs, "fp8_block", len(slots), hq, hkv, 128, 64, bs, nb, max_position=9100,
                          interleaved=hkv == 3, slots=slots, positions=pos)
    d = Dev(c)
    assert d.call() == 0
    _check(c, d)


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("hkv,seqs,most", [(1, 71, 9), (2, 176, 3), (3, 34, 5), (8, 64, 8), (8, 200, 12), (11, 40, 8)])
def test_a_few_tokens_of_many_sequences(hkv, seqs, most, bs):
    """What a step of drafted tokens appends: runs of 1 to a few tokens, some over a page's
    end, that share out a tile's blocks."""
    r = np.random.default_rng(hkv + seqs)
    spans = [(int(h), int(n)) for h, n in zip(r.integers(0, 100, seqs), r.integers(1, most + 1, seqs))]
    slots, pos, nb = _run_of(spans, bs, hkv)
    c = rope_cases.Append(seqs + bs, "fp8_block", len(slots), 2 * hkv, hkv, 128, 96, bs, nb, max_position=128,
                          interleaved=bs == 32, slots=slots, positions=pos)
    d = Dev(c)
    assert d.call() == 0
    _check(c, d)


def _append_as_kept(c, sizes, flags):
    """A page-scaled append of rows of very different sizes (scales grow and do not): written
    are the tokens that rope_cases.kept_in_pages names."""
    c.qkv[:] = rope_cases.storage(rope_cases.values(c.qkv) * sizes[:, None].astype(np.float32), "bf16")
    w = np.where(c.live() & (c.slots < c.nb * c.bs), c.slots, -1)
    kept = np.where(rope_cases.kept_in_pages(w, c.bs), w, -1)
    c.written = lambda: kept
    d = Dev(c)
    assert d.call() == flags
    _check(c, d)


@pytest.mark.parametrize("kind", ["no slot", "padding", "bad position", "bad slot"])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("had,new,hkv", [(0, 5, 2), (3, 4, 1), (0, 40, 8), (7, 200, 3), (20, 2, 8)])
def test_tokens_that_are_not_written_inside_a_page(kind, bs, had, new, hkv):
    """They leave a page's tokens one run, with one scale: of one warp or block, in one tile
    or two, and more than one of them in a row."""
    slots, pos, nb = _run_of([(had, new), (5, 3)], bs, new)
    r = np.random.default_rng(had + new)
    at = np.sort(r.choice(np.arange(1, new), max(1, new // 6), replace=False))
    at = np.repeat(at, np.where(np.arange(len(at)) % 5 == 1, 4, 1))
    out_slot, out_pos = {"no slot": (-1, 5), "padding": (7, -1), "bad position": (7, 256), "bad slot": (nb * bs, 5)}[kind]
    slots, pos = np.insert(slots, at, out_slot), np.insert(pos, at, out_pos)
    c = rope_cases.Append(new + bs, "fp8_block", len(slots), 2, hkv, 128, 64, bs, nb, max_position=256, slots=slots,
                          positions=pos)
    flags = {"bad position": pa.PA_DEVERR_BAD_POSITION, "bad slot": pa.PA_DEVERR_BAD_SLOT}.get(kind, 0)
    _append_as_kept(c, 2.0 ** r.integers(-8, 8, len(slots)), flags)


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("seqs,steps,hkv", [(2, 2, 2), (3, 5, 8), (40, 3, 1), (90, 2, 4), (150, 4, 2)])
def test_tokens_that_come_back_to_a_page_are_refused(bs, seqs, steps, hkv):
    """Drafted tokens laid out step by step instead of sequence by sequence."""
    slots = [b * bs + 2 + s for s in range(steps) for b in range(seqs)]
    c = rope_cases.Append(seqs, "fp8_block", len(slots), 4, hkv, 128, 128, bs, seqs + 1, slots=slots,
                          positions=[2 + s for s in range(steps) for _ in range(seqs)])
    assert rope_cases.kept_in_pages(slots, bs).sum() == seqs
    _append_as_kept(c, 2.0 ** np.random.default_rng(seqs).integers(-8, 8, len(slots)), pa.PA_DEVERR_BAD_SLOT)


@pytest.mark.parametrize("first", [0, 9, 15])
@pytest.mark.parametrize("gap,refused", [(45, 0), (46, 1), (47, 2), (100, 2)])
def test_tokens_far_behind_their_page(gap, refused, first):
    """Two tokens of a page, `gap` padding tokens, two more: the third is gap + 2 behind."""
    slots = [0] * first + [16, 17] + [0] * gap + [18, 19, 33]
    pos = [-1] * first + [0, 1] + [-1] * gap + [2, 3, 0]
    c = rope_cases.Append(gap, "fp8_block", len(slots), 2, 3, 128, 128, 16, 3, slots=slots, positions=pos)
    assert rope_cases.kept_in_pages(np.where(np.array(pos) < 0, -1, slots), 16).sum() == 5 - refused
    _append_as_kept(c, np.array([2.0 ** (i % 7) for i in range(len(slots))]), pa.PA_DEVERR_BAD_SLOT if refused else 0)


@pytest.mark.parametrize("factor", [1.25, 1 / 3, 1.75])
@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 2.0 ** 6])
@pytest.mark.parametrize("new,bs,hkv", [(1, 16, 8), (1, 32, 3), (7, 16, 8), (20, 32, 2), (9, 16, 1)])
def test_pages_that_go_on_under_any_scale(new, bs, hkv, size, factor):
    """Old scales that are no powers of two: kept, rows are divided by them; outgrown, the
    rows of the page come to the new one by the rounded quotient."""
    slots, pos, nb = _run_of([(5, new), (11, new)], bs, new)
    c = rope_cases.Append(new + bs, "fp8_block", len(slots), 2, hkv, 128, 96, bs, nb, slots=slots, positions=pos)
    for s in (c.k_scales, c.v_scales):
        s *= np.float32(factor)
    c.qkv[:] = rope_cases.storage(rope_cases.values(c.qkv) * np.float32(size), "bf16")
    d = Dev(c)
    assert d.call() == 0
    _check(c, d)


def _special_rows(tokens, hkv):
    """A head each of zeros, subnormals, infinities, NaN, the largest finite values."""
    x = np.random.default_rng(tokens).standard_normal((tokens, 2 * hkv, 128)).astype(np.float32)
    for base in (0, hkv):
        x[:, base] = 0.0
        x[:, base + 1] = 1e-39
        x[tokens // 3, base + 2, 5], x[tokens // 2, base + 2, 70], x[-1, base + 2, 7] = np.inf, -np.inf, np.nan
        x[:, base + 3] = 3.3e38
        x[:, base + 4] = -1e-30
        x[:, base + 5, 1:] = np.nan
        x[:, base + 6] = np.inf
    return x


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("each", [1, 2, 16])
@pytest.mark.parametrize("rot", [128, 48])
def test_special_values_that_turn(inter, each, rot):
    """The special values through the rotation, `each` tokens a call into one page."""
    hkv, bs, nb = 8, 16, 2
    rows = _special_rows(16, hkv)
    state = None
    for at in range(0, 16, each):
        c = rope_cases.Append(at, "fp8_block", each, 0, hkv, 128, rot, bs, nb, interleaved=inter,
                              slots=[16 + at + i for i in range(each)], positions=[3 + at + i for i in range(each)])
        c.qkv[:] = rope_cases.storage(rows[at:at + each].reshape(each, -1), "bf16")
        if state is not None:
            c.k_cache, c.k_scales, c.v_cache, c.v_scales = state
        d = Dev(c)
        pa.pa_rope_and_cache_fp8_block(None, None, d.k, d.v, d.kc, d.vc, d.slots, d.pos, d.table, *d.scale,
                                       interleaved=inter, device_errors=d.errs)
        assert pa.pa_read_device_errors(d.errs) == 0
        with np.errstate(all="ignore"):
            oracle.page_scale_append(c.rotated32(c.k), c.slots, c.k_cache, c.k_scales)
            oracle.page_scale_append(rope_cases.values(c.v), c.slots, c.v_cache, c.v_scales)
        for cache, s, got, gs in ((c.k_cache, c.k_scales, d.kc, d.scale[0]), (c.v_cache, c.v_scales, d.vc, d.scale[1])):
            np.testing.assert_array_equal(storage_to_host(gs, "f32"), s)
            g = storage_to_host(got, "fp8")
            nan = (cache & 0x7F) == 0x7F
            np.testing.assert_array_equal(g[~nan], cache[~nan])
            assert np.all((g[nan] & 0x7F) == 0x7F)
        state = c.k_cache, c.k_scales, c.v_cache, c.v_scales
