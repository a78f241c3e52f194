"""The prompt attention on the GPU against the oracle; prefill_cases.Prompts.bar has the
error bars."""
import numpy as np
import pytest
import torch

import paged_kv_cache_190_gb300 as pa
from fp4_cases import shifted
from gpu_helpers import DEV, out_as_f64, to_dev
from prefill_cases import Prompts
from rope_cases import storage, values

pytestmark = pytest.mark.gpu


class Dev:
    def __init__(self, c):
        self.c = c
        bf = c.dtype == "bf16"
        self.q, self.kc, self.vc = (to_dev(x, bf) for x in (c.q, c.k_cache, c.v_cache))
        self.tables, self.lens, self.starts = to_dev(c.tables), to_dev(c.lens), to_dev(c.starts)
        self.out = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device=DEV)
        self.errs = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(self, out=None, **kw):
        c = self.c
        kw = dict(max_context_len=int(c.lens.max()), window=c.window, sinks=c.sinks, device_errors=self.errs) | kw
        return pa.pa_prefill(self.out if out is None else out, self.q, self.kc, self.vc, self.tables, self.lens,
                             self.starts, c.scale, c.hkv, **kw)

    def errors(self):
        return pa.pa_read_device_errors(self.errs)


def check(c, got):
    want, parts = c.want()
    got, mine = out_as_f64(got), c.mine()
    assert (got[~mine] == 7.0).all(), "a row of no sequence was written"
    bar = c.bar(want, parts)[mine]
    err = np.abs(got[mine] - want[mine])
    assert np.all(err <= bar), f"error {np.nanmax(err / bar):.2f} of its bar, {np.isnan(err).sum()} NaN"


# (dtype, Hq, Hkv, D, bs)
KINDS = [("bf16", 4, 4, 128, 16), ("bf16", 8, 2, 128, 16), ("bf16", 8, 1, 128, 32), ("bf16", 4, 2, 64, 16),
         ("bf16", 3, 3, 64, 32), ("f32", 4, 4, 64, 16), ("f32", 8, 2, 128, 32), ("f32", 8, 1, 64, 16)]


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", KINDS)
def test_one_sequence_of_each_length(dtype, hq, hkv, d, bs):
    """From one token over the borders of pages, steps and tiles."""
    for n in (1, 2, 15, 16, 17, 33, 127, 128, 129, 300):
        c = Prompts(n + hq, dtype, [n], [0], hq, hkv, d, bs)
        dv = Dev(c)
        dv.call()
        assert dv.errors() == 0
        check(c, dv.out)


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 3), (100, 0), (130, 40), (300, 140), (5000, 2)])
def test_ragged_batches(dtype, hq, hkv, d, bs, window, sinks):
    new = [1, 0, 70, 129, 3, 400, 16, 31]
    had = [0, 50, 0, 200, 700, 37, 128, 1]
    c = Prompts(hq + bs + window, dtype, new, had, hq, hkv, d, bs, window, sinks, before=2, behind=3)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 2, 128, 16), (8, 1, 128, 32), (4, 4, 64, 16), (1, 1, 128, 16), (32, 8, 128, 16)])
@pytest.mark.parametrize("new,had", [([1], [5000]), ([64, 3, 200], [3000, 7000, 0]), ([130], [20000]),
                                     ([700, 1, 0, 33], [900, 600, 700, 5000])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 70)])
def test_few_rows_of_long_contexts(hq, hkv, d, bs, new, had, window, sinks):
    """Items too few to fill the GPU: their keys are cut into shares and joined."""
    c = Prompts(hq + sum(had), "bf16", new, had, hq, hkv, d, bs, window, sinks, before=1, behind=2)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)
    again = torch.full_like(dv.out, 7.0)
    size = pa.pa_prefill_workspace_size(c.rows, len(new), hq, hkv, d)
    dv.call(again, workspace=torch.full((size,), 0x7F, dtype=torch.uint8, device=DEV))
    assert torch.equal(again.view(torch.int16), dv.out.view(torch.int16)), "not the same bits twice"


def test_workspace_size():
    f = pa.pa_prefill_workspace_size
    assert f(0, 0, 8, 8, 128) >= 256 and f(1000, 3, 32, 8, 128) >= f(1000, 3, 8, 8, 128) >= f(10, 3, 8, 8, 128)
    c = Prompts(1, "bf16", [40], [10], 8, 2, 128, 16)
    dv = Dev(c)
    with pytest.raises(pa.PaError):
        dv.call(workspace=torch.empty(f(c.rows, 1, 8, 2, 128) - 1, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        dv.call(prepare=True)


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", KINDS)
def test_many_short_prompts(dtype, hq, hkv, d, bs):
    """More sequences than a pass of the plan, empty ones among them."""
    r = np.random.default_rng(5)
    new, had = r.integers(0, 4, 1300), r.integers(0, 20, 1300)
    c = Prompts(6, dtype, new, had, hq, hkv, d, bs, before=1, behind=1)
    dv = Dev(c)
    dv.call(max_context_len=2000 if c.tables.shape[1] * bs >= 2000 else int(c.lens.max()))
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", [("bf16", 8, 1, 128, 16), ("bf16", 2, 2, 64, 32), ("f32", 4, 4, 64, 16)])
def test_prompts_that_fill_the_gpu(dtype, hq, hkv, d, bs):
    """Several rounds of items of every length, the last of them incomplete."""
    c = Prompts(7, dtype, [2300, 500, 1800, 64, 1], [0, 700, 100, 64, 900], hq, hkv, d, bs)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", [("bf16", 8, 2, 128, 16), ("bf16", 4, 2, 64, 32), ("f32", 4, 2, 64, 16)])
def test_buffers_aligned_to_no_more_than_16_bytes(dtype, hq, hkv, d, bs):
    c = Prompts(12, dtype, [140, 3, 70], [0, 50, 200], hq, hkv, d, bs)
    dv = Dev(c)
    dv.q, dv.kc, dv.vc, dv.out = (shifted(x, 16) for x in (dv.q, dv.kc, dv.vc, dv.out))
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


def _growing(c, factor):
    """K rows whose scores grow (or fall) with the position, past any fixed reference."""
    k = values(c.k_cache).astype(np.float32)
    for b, L in enumerate(c.lens):
        t = np.arange(int(L))
        ok = (c.tables[b][t // c.bs] >= 0) & (c.tables[b][t // c.bs] < c.nb)
        t = t[ok]
        # along the mean of the sequence's own q
        rows = values(c.q)[c.starts[b]:c.starts[b + 1]]
        if len(rows) == 0:
            continue
        dirn = rows.mean(0).reshape(c.hkv, -1, rows.shape[-1]).mean(1)
        k[c.tables[b][t // c.bs], :, t % c.bs] = dirn[None] * (factor * t / max(1, L))[:, None, None]
    c.k_cache = storage(k, c.dtype)


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", KINDS)
@pytest.mark.parametrize("factor", [400.0, -400.0, 3000.0])
def test_scores_that_grow_along_the_context(dtype, hq, hkv, d, bs, factor):
    """The first step's maximum is no reference for the last step's scores."""
    c = Prompts(8, dtype, [300, 5], [200, 600], hq, hkv, d, bs)
    q = values(c.q).astype(np.float32)
    q[:] = np.abs(q)                                          # one direction for all rows: scores of one sign
    c.q = storage(q, dtype)
    _growing(c, factor)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", [("bf16", 4, 2, 128, 16), ("f32", 4, 2, 64, 16)])
def test_special_values(dtype, hq, hkv, d, bs):
    """A NaN in a row of q, an infinite key and a NaN key reach the rows that see them, and no others."""
    c = Prompts(9, dtype, [40, 30], [10, 0], hq, hkv, d, bs)
    q, k = values(c.q).astype(np.float32), values(c.k_cache).astype(np.float32)
    q[3, 1, 5] = np.nan
    at = c.tables[1][1], slice(None), 20 % bs                 # sequence 1, position 20 (page 1)
    k[at[0], 0, at[2]] = np.nan
    k[at[0], 1, at[2]] = np.float32(3e38)
    c.q, c.k_cache = storage(q, dtype), storage(k, dtype)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    got = out_as_f64(dv.out)
    nan = np.isnan(got).all(-1)
    want = np.zeros_like(nan)
    want[3, 1] = True
    page1 = c.starts[1] + 16
    first = c.starts[1] + 16 + (20 % bs)                      # the key's own row and those behind it
    want[first:c.starts[2], :hq // 2] = True
    assert (nan[:, :hq // 2] == want[:, :hq // 2]).all()
    assert not np.isnan(got[:page1][~want[:page1]]).any()
    assert np.isfinite(got[:c.starts[1], hq // 2:]).all()


def test_refused_data():
    c = Prompts(10, "bf16", [20, 30, 10], [0, 40, 5], 4, 2, 128, 16)
    ref = Dev(c)
    ref.call()
    # a page that is none, in the middle of sequence 1: its tokens are not seen
    dv = Dev(c)
    dv.tables[1, 2] = c.nb
    dv.call()
    assert dv.errors() == pa.PA_DEVERR_BAD_BLOCK
    k, v = (values(x).astype(np.float64) for x in (c.k_cache, c.v_cache))
    t = np.array([x for x in range(70) if x // 16 != 2])
    kk, vv = (x[c.tables[1][t // 16], :, t % 16] for x in (k, v))
    qq = values(c.q).astype(np.float64)[20:50]
    for j in (0, 29):
        see = t <= 40 + j
        for i in range(4):
            s = c.scale * (kk[see][:, i // 2] @ qq[j, i])
            w = np.exp(s - s.max())
            np.testing.assert_allclose(out_as_f64(dv.out)[20 + j, i], (w / w.sum()) @ vv[see][:, i // 2], atol=0.03)
    same = torch.equal(dv.out[:20], ref.out[:20]) and torch.equal(dv.out[50:], ref.out[50:])
    assert same, "other sequences' rows changed"
    # a length that is none: clamped
    for bad in (-1, 10 ** 6):
        dv = Dev(c)
        dv.lens[2] = bad
        dv.call(max_context_len=70)
        assert dv.errors() & pa.PA_DEVERR_BAD_LENGTH
        assert torch.equal(dv.out[:50], ref.out[:50])
    # fewer tokens than new ones: the rows before the first token see nothing
    dv = Dev(c)
    dv.lens[0] = 15
    dv.call()
    assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH and bool((dv.out[:5] == 0).all()) and bool((dv.out[5:20] != 0).any())
    # starts that leave the rows or decrease
    for starts in ([-1, 20, 50, 60], [0, 20, 50, 61], [0, 50, 20, 60], [0, 60, 0, 60]):
        dv = Dev(c)
        dv.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
        dv.call()
        assert dv.errors() & pa.PA_DEVERR_BAD_LENGTH
    ref.call()
    assert ref.errors() == 0


def test_rows_that_see_nothing():
    c = Prompts(11, "bf16", [5, 7], [0, 0], 4, 2, 64, 16)
    dv = Dev(c)
    dv.lens.zero_()
    dv.call(max_context_len=0)
    assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH and bool((dv.out == 0).all())
    dv = Dev(c)
    dv.starts.zero_()                                        # no new tokens at all
    dv.call()
    assert dv.errors() == 0 and bool((dv.out == 7).all())


@pytest.mark.parametrize("new,had", [([300, 40], [0, 100]), ([64], [9000])])
def test_captured_and_replayed(new, had):
    """One graph, other lengths, pages and values at each replay; the same bits as a call."""
    c = Prompts(12, "bf16", new, had, 8, 2, 128, 16)
    dv = Dev(c)
    most = int(c.lens.max())
    ws = torch.empty(pa.pa_prefill_workspace_size(c.rows, len(new), 8, 2, 128), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        dv.call(workspace=ws)
        with torch.cuda.graph(g, stream=s):
            dv.call(workspace=ws, max_context_len=most)
            dv.call(workspace=ws, max_context_len=most)
    s.synchronize()
    for cut in (0, 1, 37):
        dv.lens.copy_(torch.from_numpy(c.lens - cut))
        dv.starts[-1] = int(c.starts[-1]) - cut              # fewer new tokens of the last sequence too
        dv.q.copy_(dv.q.flip(0))
        dv.out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        again = torch.full_like(dv.out, 7.0)
        dv.call(again, max_context_len=most)
        assert torch.equal(again, dv.out)
        dv.errors()


def test_two_streams_at_once():
    cs = [Prompts(13 + i, "bf16", [400, 30], [0, 3000], 8, 2, 128, 16) for i in range(2)]
    dvs = [Dev(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        for dv, s in zip(dvs, streams):
            dv.call(stream=s)                                # each call's own workspace
    torch.cuda.synchronize()
    for c, dv in zip(cs, dvs):
        assert dv.errors() == 0
        check(c, dv.out)


def test_prepared_call():
    c = Prompts(15, "bf16", [50], [100], 8, 2, 128, 16)
    dv = Dev(c)
    ws = torch.empty(pa.pa_prefill_workspace_size(c.rows, 1, 8, 2, 128), dtype=torch.uint8, device=DEV)
    call = dv.call(workspace=ws, prepare=True)
    call()
    call()
    assert dv.errors() == 0
    check(c, dv.out)


def test_python_refusals():
    c = Prompts(16, "bf16", [50], [100], 8, 2, 128, 16)
    dv = Dev(c)
    for name, bad, err in (("q", dv.q.float(), TypeError), ("q", dv.q[:, ::2], ValueError), ("kc", dv.kc[:, :1], ValueError),
                           ("tables", dv.tables.long(), TypeError), ("lens", dv.lens[:0], ValueError),
                           ("starts", dv.starts[:1], ValueError), ("starts", dv.starts.cpu(), ValueError),
                           ("tables", dv.tables[0], ValueError)):
        other = Dev(c)
        setattr(other, name, bad)
        with pytest.raises(err):
            other.call()
    with pytest.raises(ValueError):
        dv.call(out=dv.out[:-1])
    with pytest.raises(TypeError):
        dv.call(out=dv.out.float())
    with pytest.raises(pa.PaError):
        dv.call(window=0, sinks=3)
    assert dv.errors() == 0


@pytest.mark.parametrize("limit", [0, 64])
@pytest.mark.parametrize("d,new,had", [(128, [600, 33], [0, 900]), (64, [100], [6000]), (128, [20], [0])])
def test_expired_waits_report_and_leave_the_context_usable(limit, d, new, had):
    c = Prompts(17, "bf16", new, had, 8, 2, d, 16)
    dv = Dev(c)
    try:
        pa.pa_debug_set_wait_limit(limit)
        for _ in range(3):
            dv.call()
        flags = dv.errors()                                  # synchronises: the kernel returned
    finally:
        pa.pa_debug_set_wait_limit(-1)
    assert flags & ~pa.PA_DEVERR_TIMEOUT == 0 and (limit or flags)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


def test_pages_past_32_bits():
    """A pool of more than 2^32 bytes whose last pages hold the context."""
    hkv, d, bs = 8, 128, 16
    nb = (1 << 32) // (hkv * bs * d * 2) + 40
    c = Prompts(18, "bf16", [70], [200], 16, hkv, d, bs)
    dv = Dev(c)
    pools = []
    for small in (dv.kc, dv.vc):
        big = torch.empty(nb, hkv, bs, d, dtype=torch.bfloat16, device=DEV)
        big[nb - c.nb:].copy_(small)
        pools.append(big)
    ok = (dv.tables >= 0) & (dv.tables < c.nb)
    dv.tables = torch.where(ok, dv.tables + (nb - c.nb), -1)
    dv.kc, dv.vc = pools
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)
