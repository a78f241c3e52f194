"""The windowed decode and the decode over page-scaled e4m3 pools on the GPU against the
oracle; span_cases.Decode.bar has the error bars."""
import types

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
from gpu_helpers import DEV, out_as_f64, to_dev
from span_cases import Decode

pytestmark = pytest.mark.gpu


class Dev:
    def __init__(self, c):
        self.c = c
        bf = c.dtype != "f32"
        q = c.q if c.q_len > 1 else c.q[:, 0]
        self.q = to_dev(q, bf)
        self.kc, self.vc = (to_dev(x, c.dtype == "bf16") for x in (c.k_cache, c.v_cache))
        self.tables, self.lens = to_dev(c.tables), to_dev(c.lens)
        self.scales = tuple(to_dev(s) for s in c.scales)
        self.out = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device=DEV)
        self.errs = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(self, out=None, **kw):
        c = self.c
        out = self.out if out is None else out
        kw = dict(max_context_len=int(c.lens.max()), window=c.window, sinks=c.sinks, device_errors=self.errs) | kw
        if c.dtype == "fp8":
            return pa.pa_decode_fp8_block(out, self.q, self.kc, self.vc, self.tables, self.lens, c.scale,
                                          *self.scales, c.hkv, **kw)
        return pa.pa_decode_window(out, self.q, self.kc, self.vc, self.tables, self.lens, c.scale, c.hkv, **kw)

    def errors(self):
        return pa.pa_read_device_errors(self.errs)


def check(c, got, rows=None):
    want, parts = c.want()
    got = out_as_f64(got).reshape(want.shape)
    bar = c.bar(want, parts)
    if rows is not None:
        got, want, bar = got[rows], want[rows], bar[rows]
    worst = np.max(np.abs(got - want) / bar)
    assert np.all(np.abs(got - want) <= bar), f"error {worst:.2f} of its bar"


# (dtype, q_len, Hq, Hkv, D, bs)
KINDS = [("bf16", 1, 8, 8, 128, 16), ("bf16", 1, 8, 2, 128, 32), ("bf16", 2, 8, 2, 64, 16), ("bf16", 1, 6, 3, 64, 32),
         ("bf16", 8, 2, 2, 128, 16), ("f32", 1, 8, 8, 64, 16), ("f32", 1, 8, 1, 128, 16), ("f32", 4, 2, 1, 64, 32),
         ("f32", 2, 3, 3, 128, 32), ("fp8", 1, 32, 8, 128, 16), ("fp8", 1, 3, 3, 128, 32), ("fp8", 2, 8, 2, 128, 16),
         ("fp8", 8, 4, 4, 128, 32), ("fp8", 1, 8, 1, 128, 16)]
WINDOWS = [(0, 0), (1, 0), (1, 1), (16, 4), (33, 0), (64, 17), (100, 70), (5000, 2)]


@pytest.mark.parametrize("dtype,q_len,hq,hkv,d,bs", KINDS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_small_calls(dtype, q_len, hq, hkv, d, bs, window, sinks):
    lens = [q_len, q_len + 1, 15 + q_len, 16 + q_len, 33 + q_len, 97, 131, 300]
    c = Decode(len(dtype) + q_len + hq + bs + window, dtype, lens, q_len, hq, hkv, d, bs, window, sinks, spread=3)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("dtype,q_len,hq,hkv,d,bs", [
    ("bf16", 1, 16, 8, 128, 16), ("bf16", 2, 8, 2, 128, 32), ("bf16", 1, 3, 3, 64, 16), ("f32", 1, 8, 8, 64, 16),
    ("f32", 8, 1, 1, 128, 16), ("fp8", 1, 16, 8, 128, 16), ("fp8", 1, 16, 16, 128, 16), ("fp8", 2, 8, 2, 128, 32),
    ("fp8", 8, 1, 1, 128, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 4), (90, 33)])
def test_large_calls_in_shares(dtype, q_len, hq, hkv, d, bs, window, sinks):
    """Enough work that it goes out in equal shares, with sequences cut anywhere, several
    in a share, and one that spans many shares."""
    r = np.random.default_rng(hq + d)
    lens = [int(x) for x in r.integers(q_len, 400, 37)] + [6000, q_len, 3000]
    c = Decode(hq + hkv + bs, dtype, lens, q_len, hq, hkv, d, bs, window, sinks, spread=2)
    dv = Dev(c)
    # the bound that the caller gives may be far above the lengths
    width = 120000 // bs
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    tables[:, :dv.tables.shape[1]] = dv.tables
    dv.tables = tables
    dv.call(max_context_len=120000, window=window or 0)
    assert dv.errors() == 0
    check(c, dv.out)
    again = torch.empty_like(dv.out)
    dv.call(again, max_context_len=120000, workspace=torch.full((64 << 20,), 0x7F, dtype=torch.uint8, device=DEV))
    assert torch.equal(again.view(torch.int16), dv.out.view(torch.int16)), "not the same bits twice"


@pytest.mark.parametrize("dtype,q_len,hq,hkv,d,bs", [
    ("bf16", 1, 8, 8, 128, 16), ("bf16", 4, 6, 3, 64, 32), ("f32", 2, 2, 2, 64, 16), ("f32", 1, 1, 1, 128, 32),
    ("fp8", 1, 8, 8, 128, 16), ("fp8", 2, 4, 4, 128, 32), ("fp8", 1, 3, 3, 128, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (17, 50)])
def test_more_sequences_than_clusters_fit(dtype, q_len, hq, hkv, d, bs, window, sinks):
    """More sequences than the GPU has SMs: shares with many short segments each, empty ones
    among them, cut anywhere."""
    r = np.random.default_rng(hq + bs)
    lens = [int(x) for x in r.integers(q_len, 150, 190)] + [0, 0, 700, q_len]
    r.shuffle(lens)
    c = Decode(hkv + bs, dtype, lens, q_len, hq, hkv, d, bs, window, sinks, spread=2)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)
    again = torch.empty_like(dv.out)
    dv.call(again, workspace=torch.full((64 << 20,), 0x7F, dtype=torch.uint8, device=DEV))
    assert torch.equal(again.view(torch.int16), dv.out.view(torch.int16)), "not the same bits twice"


@pytest.mark.parametrize("dtype,window", [("bf16", 0), ("bf16", 9), ("fp8", 0), ("f32", 5)])
def test_thousands_of_short_sequences(dtype, window):
    """More sequences in a share than a warp's lanes hold lengths of, several for each
    thread of the pass over them."""
    r = np.random.default_rng(30)
    c = Decode(31, dtype, [int(x) for x in r.integers(0, 24, 6001)], 1, 1, 1, 64 if dtype == "bf16" else 128, 16,
               window, 2 if window else 0, spread=1)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("dtype,q_len,hq,hkv,B,longest", [
    ("fp8", 1, 32, 8, 12, 900), ("fp8", 2, 32, 8, 30, 300), ("fp8", 1, 8, 8, 100, 200), ("fp8", 8, 8, 8, 5, 2000),
    ("bf16", 1, 32, 8, 12, 900), ("bf16", 2, 32, 8, 30, 300), ("bf16", 1, 8, 8, 120, 100), ("bf16", 8, 8, 8, 3, 3000),
    ("f32", 1, 32, 8, 6, 700), ("f32", 8, 8, 8, 40, 60), ("f32", 1, 16, 16, 9, 250)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (120, 5)])
def test_middling_calls(dtype, q_len, hq, hkv, B, longest, window, sinks):
    """Between one sequence and a full GPU: clusters of every size and head group."""
    r = np.random.default_rng(B)
    lens = [int(x) for x in r.integers(q_len, longest, B - 1)] + [longest]
    c = Decode(B + q_len, dtype, lens, q_len, hq, hkv, 128, 16, window, sinks, spread=2)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


def test_nothing_to_attend_to():
    c = Decode(32, "bf16", [5, 9], 1, 4, 2, 64, 16)
    dv = Dev(c)
    dv.lens.zero_()
    dv.call(max_context_len=0)
    assert dv.errors() == 0 and bool((dv.out == 0).all())
    empty = dv.q[:0]
    out = pa.pa_decode_window(empty.clone(), empty, dv.kc, dv.vc, dv.tables[:0], dv.lens[:0], 1.0, 2, 9, 4)
    assert out.shape[0] == 0


def test_prepared_calls_and_a_given_stream():
    for dt in ("bf16", "fp8"):
        c = Decode(33, dt, [300, 45, 200], 1, 8, 4, 128, 16, window=64, sinks=4)
        dv = Dev(c)
        ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        call = dv.call(workspace=ws, prepare=True)
        assert isinstance(call, pa.PreparedCall)
        call()
        check(c, dv.out)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        again = torch.empty_like(dv.out)
        dv.call(again, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(again.view(torch.int16), dv.out.view(torch.int16))


def test_its_own_workspace_outlives_a_call_on_another_stream():
    """The workspace that a call allocates is not given out again while another stream's
    call still needs it: here that call runs after 4 ms of other work, while the memory that
    the current stream got meanwhile is overwritten again and again."""
    c = Decode(36, "bf16", [int(x) for x in np.random.default_rng(5).integers(1, 400, 180)], 1, 4, 4, 128, 16)
    dv = Dev(c)
    dv.call()
    nbytes = pa.pa_decode_window_workspace_size(len(c.lens), 4, 4, 128, 16, int(c.lens.max()))
    torch.cuda.synchronize()
    side, again, busy = torch.cuda.Stream(), torch.empty_like(dv.out), torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(8_000_000)
    dv.call(again, stream=side)
    other = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
    busy.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(busy):
        for _ in range(4000):
            other.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), dv.out.view(torch.int16))


def test_two_streams_at_once():
    """Two large calls in flight together, a workspace each, over and over."""
    cs = [Decode(34 + i, dt, [int(x) for x in np.random.default_rng(i).integers(1, 400, 180)], 1, 4, 4, 128, 16)
          for i, dt in enumerate(("bf16", "fp8"))]
    dvs = [Dev(c) for c in cs]
    for dv in dvs:
        dv.call()
        dv.ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        dv.side = torch.cuda.Stream()
        dv.side.wait_stream(torch.cuda.current_stream())
    want = [dv.out.clone() for dv in dvs]
    outs = [[torch.empty_like(dv.out) for dv in dvs] for _ in range(20)]
    torch.cuda.synchronize()
    for o in outs:
        for dv, x in zip(dvs, o):
            dv.call(x, workspace=dv.ws, stream=dv.side)
    torch.cuda.synchronize()
    for o in outs:
        for w, x in zip(want, o):
            assert torch.equal(w.view(torch.int16), x.view(torch.int16))


def test_one_long_sequence_over_all_shares():
    c = Decode(3, "fp8", [50000], 1, 8, 8, 128, 16, spread=1)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)
    c = Decode(4, "bf16", [40001, 7], 1, 2, 2, 64, 32, window=39000, sinks=5)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_empty_sequences_and_refused_lengths(dtype, big):
    d = 128
    lens = [0, 40, 0, 3, 70] + [0] * 9
    c = Decode(5, dtype, lens, 1, 4, 2, d, 16, window=30, sinks=2)
    dv = Dev(c)
    most = 200000 if big else 80
    if big:
        dv.tables = torch.nn.functional.pad(dv.tables, (0, 200000 // 16 - dv.tables.shape[1]), value=-1)
    else:
        dv.tables = torch.nn.functional.pad(dv.tables, (0, 6), value=-1)
    kw = dict(max_context_len=most, window=30 if not big else 30)
    dv.call(**kw)
    assert dv.errors() == 0
    check(c, dv.out)
    assert bool((dv.out[[0, 2]] == 0).all())
    dv.lens[0] = -5
    dv.call(**kw)
    assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH
    check(c, dv.out)


def test_length_past_the_bound_is_flagged_and_cut():
    c = Decode(6, "bf16", [48, 48], 1, 2, 2, 64, 16)
    dv = Dev(c)
    dv.lens[1] = 100
    dv.call(max_context_len=48)
    assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH
    check(c, dv.out)


def test_fewer_tokens_than_new_ones():
    c = Decode(7, "bf16", [2, 40], 4, 2, 2, 128, 16, window=9)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH
    assert bool((dv.out[0, :2] == 0).all())
    check(c, dv.out)


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("f32", 16), ("fp8", 16), ("fp8", 32)])
def test_missing_pages_are_flagged_and_left_out(dtype, bs):
    """A bad entry inside the window: its tokens drop out as if they were not there."""
    c = Decode(8, dtype, [200, 200, 64], 1, 4, 2, 128, bs, window=100, sinks=3)
    bad = 150 // bs
    dv = Dev(c)
    dv.tables[1, bad] = c.nb + 3
    dv.call()
    assert dv.errors() == pa.PA_DEVERR_BAD_BLOCK
    check(c, dv.out, rows=[0, 2])
    got = out_as_f64(dv.out)[1]
    page = [p for p in range(200) if p < 3 or (p >= 100 and p // bs != bad)]
    from rope_cases import values
    if dtype == "fp8":
        k, v = (oracle.E4M3_VALUES[x] * s[:, :, None, None].astype(np.float64)
                for x, s in zip((c.k_cache, c.v_cache), c.scales))
    else:
        k, v = (values(x).astype(np.float64) for x in (c.k_cache, c.v_cache))
    for i in range(4):
        kk, vv = (np.stack([x[c.tables[1, p // bs], i // 2, p % bs] for p in page]) for x in (k, v))
        s = c.scale * kk @ values(c.q)[1, 0, i].astype(np.float64)
        w = np.exp(s - s.max())
        w /= w.sum()
        assert np.max(np.abs(got[i] - w @ vv)) <= (1e-5 if dtype == "f32" else 2e-2)


def test_no_window_agrees_with_the_full_decode():
    c = Decode(9, "bf16", [700, 33, 1], 1, 16, 4, 128, 16)
    dv = Dev(c)
    dv.call()
    full = torch.empty_like(dv.out)
    pa.pa_decode(full, dv.q, dv.kc, dv.vc, dv.tables, dv.lens, c.scale, c.hkv, 700, device_errors=dv.errs)
    assert dv.errors() == 0
    check(c, dv.out)
    check(c, full)


@pytest.mark.parametrize("dtype,q_len,hq,hkv", [("bf16", 1, 8, 8), ("fp8", 1, 16, 8), ("f32", 2, 8, 8), ("bf16", 2, 8, 2),
                                                ("fp8", 4, 3, 3)])
@pytest.mark.parametrize("seqs,most", [(1, 700), (2, 300), (3, 1500), (7, 700), (10, 1500), (12, 700), (20, 700), (24, 1500),
                                       (45, 700)])
def test_sequences_split_over_any_number_of_blocks(dtype, q_len, hq, hkv, seqs, most):
    """The longest sequence over 1 to 8 blocks, the others over as many, some with less than
    a tile for each."""
    lens = np.random.default_rng(seqs).integers(q_len, most // 2, seqs)
    lens[0], lens[-1] = q_len, most
    c = Decode(seqs, dtype, lens, q_len, hq, hkv, 128, 16)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("dtype,seqs,q_len,hq,hkv", [("bf16", 232, 2, 32, 8), ("fp8", 294, 8, 4, 4), ("f32", 300, 1, 4, 4),
                                                     ("bf16", 512, 1, 8, 8), ("f32", 232, 2, 16, 4), ("fp8", 700, 1, 4, 1)])
def test_more_short_sequences_than_blocks_fit(dtype, seqs, q_len, hq, hkv):
    lens = np.random.default_rng(seqs).integers(q_len, 41, seqs)
    c = Decode(seqs, dtype, lens, q_len, hq, hkv, 128, 16, window=30, sinks=2)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("norm", [1e-30, 2.0 ** -20, 2.0 ** 12, 0.0])
def test_first_pages_with_values_of_another_size(norm):
    """V rows of the first page far smaller (as first tokens' are) or larger than the rest."""
    c = Decode(10, "fp8", [16, 20, 333], 1, 8, 2, 128, 16, first_norm=norm)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


def test_wide_scores():
    for dtype in ("bf16", "f32", "fp8"):
        c = Decode(11, dtype, [400, 77], 1, 8, 4, 128, 16, window=150, sinks=4, std=4.0)
        dv = Dev(c)
        dv.call()
        check(c, dv.out)


@pytest.mark.parametrize("dtype,lens", [("bf16", [300, 900]), ("fp8", [300, 900]), ("f32", [300, 900]),
                                        ("bf16", [3000] * 60), ("fp8", [5000] * 60), ("bf16", [300] * 170),
                                        ("fp8", [300] * 170), ("f32", [100] * 170)])
@pytest.mark.parametrize("polls", [0, 40])
def test_expired_waits_report_and_leave_the_context_usable(dtype, lens, polls):
    B, hkv, d, bs = len(lens), 8, 128, 16
    r = torch.Generator(device=DEV).manual_seed(1)
    width = -(-max(lens) // bs)
    nb = 512
    tables = torch.randint(0, nb, (B, width), generator=r, device=DEV, dtype=torch.int32)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    q = torch.randn(B, 8, d, generator=r, device=DEV).to(dt)
    kc = torch.randn(nb, hkv, bs, d, generator=r, device=DEV)
    vc = torch.randn(nb, hkv, bs, d, generator=r, device=DEV)
    kc, vc = (x.to(torch.float8_e4m3fn) if dtype == "fp8" else x.to(dt) for x in (kc, vc))
    one = torch.ones(nb, hkv, device=DEV)
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call():
        out = torch.empty_like(q)
        if dtype == "fp8":
            pa.pa_decode_fp8_block(out, q, kc, vc, tables, n, d ** -0.5, one, one, hkv, max(lens), device_errors=errs)
        else:
            pa.pa_decode_window(out, q, kc, vc, tables, n, d ** -0.5, hkv, max(lens), 0, device_errors=errs)
        return out

    want = call()
    assert pa.pa_read_device_errors(errs) == 0
    try:
        pa.pa_debug_set_wait_limit(polls)
        call()
        flags = pa.pa_read_device_errors(errs)
    finally:
        pa.pa_debug_set_wait_limit(-1)
    assert flags == pa.PA_DEVERR_TIMEOUT if polls == 0 else flags & ~pa.PA_DEVERR_TIMEOUT == 0
    assert torch.equal(call().view(torch.int16), want.view(torch.int16))
    assert pa.pa_read_device_errors(errs) == 0


def test_pools_past_32_bit_offsets():
    """Pages at the far end of pools of more than 2^32 bytes."""
    hkv, bs, d = 32, 16, 128
    nb = (1 << 32) // (hkv * bs * d) + 9
    kc = torch.zeros(nb, hkv, bs, d, dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    ks = torch.full((nb, hkv), float("nan"), device=DEV)
    vs = ks.clone()
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(2, 40, hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    page = torch.tensor([nb - 1, nb - 5, nb - 3], device=DEV)
    slots = (page[:, None] * bs + torch.arange(bs, device=DEV)).flatten()[:40]
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rope_and_cache_fp8_block(None, None, x[0], x[1], kc, vc, slots, None, None, ks, vs, device_errors=errs)
    q = torch.randn(1, hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.empty_like(q)
    pa.pa_decode_fp8_block(out, q, kc, vc, page.int()[None], torch.tensor([40], dtype=torch.int32, device=DEV),
                           d ** -0.5, ks, vs, hkv, 48, device_errors=errs)
    assert pa.pa_read_device_errors(errs) == 0
    s = torch.einsum("hd,thd->ht", q[0].double(), x[0].double()) * d ** -0.5
    want = torch.einsum("ht,thd->hd", s.softmax(-1), x[1].double())
    # e4m3 keys and values: 2^-4 of each V element, and of each key's product
    dots = torch.einsum("hd,thd->ht", q[0].double().abs(), x[0].double().abs()).amax(-1) * d ** -0.5 * 2.0 ** -4
    mag = torch.einsum("ht,thd->hd", s.softmax(-1), x[1].double().abs())
    assert bool(((out[0].double() - want).abs() <= (2.0 ** -4 + 2.0 ** -7 + 2 * dots[:, None]) * mag + 2.0 ** -8).all())


def test_other_stream_and_captured_graphs():
    """Calls on a stream of their own, captured with a workspace each, replayed with other
    lengths, in turn and against eager calls."""
    cs = [Decode(12 + i, dt, [300, 45, 200], 1, 8, 4, 128, 16, window=64, sinks=4)
          for i, dt in enumerate(("bf16", "fp8", "f32"))]
    dvs = [Dev(c) for c in cs]
    for dv in dvs:
        dv.call()
    eager = [dv.out.clone() for dv in dvs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for dv in dvs:
            dv.ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
            dv.call(workspace=dv.ws)
        side.synchronize()
        for dv in dvs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                dv.call(workspace=dv.ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(2):
        for dv in dvs:
            dv.out.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for dv, e in zip(dvs, eager):
            assert torch.equal(dv.out.view(torch.int16), e.view(torch.int16))
    # other inputs in the same buffers
    for dv in dvs:
        dv.q.copy_(dv.q.flip(0))
        dv.lens[1] = 44
    for g in reversed(graphs):
        g.replay()
    torch.cuda.synchronize()
    for dv in dvs:
        replayed = dv.out.clone()
        dv.call()
        assert torch.equal(dv.out.view(torch.int16), replayed.view(torch.int16))
        assert dv.errors() == 0


def test_refusals_of_the_python_call():
    c = Decode(15, "bf16", [20, 20], 1, 4, 2, 128, 16)
    dv = Dev(c)
    ok = dict(out=dv.out, q=dv.q, k_cache=dv.kc, v_cache=dv.vc, block_tables=dv.tables, context_lens=dv.lens,
              scale=1.0, num_kv_heads=2, max_context_len=20, window=4)
    pa.pa_decode_window(**ok)
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    for over, kind in ((dict(q=dv.q.float()), (TypeError, ValueError)), (dict(out=dv.out[:1]), ValueError),
                       (dict(k_cache=dv.kc.float()), TypeError), (dict(v_cache=dv.vc[:1]), ValueError),
                       (dict(num_kv_heads=4), ValueError), (dict(context_lens=dv.lens[:1]), ValueError),
                       (dict(block_tables=dv.tables.long()), TypeError), (dict(window=-1), pa.PaError),
                       (dict(window=0, sinks=3), pa.PaError), (dict(workspace=small), pa.PaError),
                       (dict(max_context_len=10 ** 6), pa.PaError),
                       (dict(block_tables=dv.tables.t()), ValueError), (dict(context_lens=dv.lens.cpu()), ValueError)):
        with pytest.raises(kind):
            pa.pa_decode_window(**{**ok, **over})


@pytest.mark.parametrize("q_len,hq,hkv,d,bs", [(1, 8, 8, 128, 16), (1, 8, 2, 128, 32), (2, 8, 2, 64, 16),
                                               (8, 2, 2, 128, 16), (1, 3, 3, 64, 32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
@pytest.mark.parametrize("seqs", [2, 40, 200])
def test_bf16_weights_are_not_rounded_to_bf16(q_len, hq, hkv, d, bs, window, sinks, seqs):
    """The weights reach the product with V in two bf16 parts, p = hi + lo + e: hi is within
    2^-8 of p, lo within 2^-8 of p - hi, so |e| <= 2^-16 p.  What is left of the error is the
    result's own half step, 2^-8, and the scores'.  Small scores (std 0.25) keep the scores'
    part under 2^-14; values of both signs leave results far under the sum of the magnitudes,
    where a rounding of each weight to bf16 shows."""
    r = np.random.default_rng(seqs)
    lens = [int(x) for x in r.integers(q_len, 300, seqs - 1)] + [300]
    c = Decode(50 + d, "bf16", lens, q_len, hq, hkv, d, bs, window, sinks, std=0.25)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    want, parts = c.want()
    rel = 2.0 ** -21 * d * parts["dots"][..., None] + 2.0 ** -20
    bar = 2.0 ** -8 * np.abs(want) + (2.0 ** -16 * 1.01 + rel) * parts["mag"] + 1e-37
    err = np.abs(out_as_f64(dv.out).reshape(want.shape) - want)
    assert np.all(err <= bar), f"error {np.max(err / bar):.2f} of its bar"


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_its_own_workspace_is_no_memory_that_the_current_stream_still_reads(dtype, raw):
    """Memory freed on the current stream, of which a copy is still due there, is not the
    workspace of a call on another stream."""
    c = Decode(37, dtype, [int(x) for x in np.random.default_rng(6).integers(1, 400, 180)], 1, 4, 4, 128, 16)
    dv = Dev(c)
    dv.call()
    nbytes = pa.pa_decode_window_workspace_size(len(c.lens), 4, 4, 128, 16, int(c.lens.max()))
    side, again = torch.cuda.Stream(), torch.empty_like(dv.out)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = torch.full((nbytes,), 17, dtype=torch.uint8, device=DEV)
    copied = torch.empty_like(freed)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    copied.copy_(freed)
    del freed
    dv.call(again, stream=types.SimpleNamespace(cuda_stream=side.cuda_stream) if raw else side)
    torch.cuda.synchronize()
    assert bool((copied == 17).all())
    assert torch.equal(again.view(torch.int16), dv.out.view(torch.int16))
