"""4-bit pools on the GPU: the append code for code, pages read back exactly, the decode under
fp4_cases.Decode4.bar."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
from fp4_cases import Append4, Decode4, pool, shifted
from gpu_helpers import DEV, out_as_f64, to_dev
from rope_cases import storage, values

pytestmark = pytest.mark.gpu


class DevAppend:
    def __init__(self, c):
        self.c = c
        x = to_dev(c.qkv, True).view(len(c.qkv), -1, 128)
        self.q, self.k, self.v = x[:, :c.hq], x[:, c.hq:c.hq + c.hkv], x[:, c.hq + c.hkv:]
        self.kc, self.vc = to_dev(c.k_cache), to_dev(c.v_cache)
        self.slots, self.pos, self.table = to_dev(c.slots), to_dev(c.positions), to_dev(c.cos_sin)
        self.q_out = torch.full((len(c.qkv), c.hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        self.errs = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(self, **kw):
        c = self.c
        args = (self.q_out, self.q) if c.hq else (None, None)
        pa.pa_rope_and_cache_fp4(*args, self.k, self.v, self.kc, self.vc, self.slots, self.pos, self.table,
                                 interleaved=c.interleaved, device_errors=self.errs, **kw)
        return pa.pa_read_device_errors(self.errs)


def check_append(c, dv):
    for name, want, got in zip("kv", c.want(), (dv.kc, dv.vc)):
        got = got.cpu().numpy()
        np.testing.assert_array_equal(got[..., 64:], want[..., 64:], err_msg=name + " scales")
        np.testing.assert_array_equal(oracle.unpack_rows(got), oracle.unpack_rows(want), err_msg=name)
    live = c.live()
    got = dv.q_out.float().cpu().numpy()
    assert (got[~live] == 7.0).all()
    np.testing.assert_array_equal(got[live], values(storage(c.rotated32(c.q)[live], "bf16")))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 32, 48, 80, 112, 128])
@pytest.mark.parametrize("hq,hkv,bs", [(8, 8, 16), (6, 3, 32), (8, 1, 16)])
def test_append(rot, hq, hkv, bs, interleaved):
    c = Append4(rot + hq, 45, hq, hkv, rot, bs, 5, interleaved=interleaved)
    dv = DevAppend(c)
    assert dv.call() == 0
    check_append(c, dv)


@pytest.mark.parametrize("tokens", [1, 2, 700])
def test_append_of_few_and_many_tokens(tokens):
    c = Append4(tokens, tokens, 32, 8, 128, 16, 60)
    dv = DevAppend(c)
    assert dv.call() == 0
    check_append(c, dv)


def test_append_padding_and_refused_tokens():
    slots = [3, -1, 17, 5 * 16, 40, 41, 42, 2 ** 40]
    pos = [0, 5, -1, 7, 64, 63, 2 ** 40, 9]
    c = Append4(5, 8, 4, 2, 128, 16, 5, slots=slots, positions=pos)
    dv = DevAppend(c)
    assert dv.call() == pa.PA_DEVERR_BAD_SLOT | pa.PA_DEVERR_BAD_POSITION
    check_append(c, dv)


def test_append_without_rotation_or_queries():
    c = Append4(6, 30, 4, 4, 128, 32, 4)
    dv = DevAppend(c)
    pa.pa_rope_and_cache_fp4(None, None, dv.k, dv.v, dv.kc, dv.vc, dv.slots, None, None, device_errors=dv.errs)
    c.cos_sin = c.cos_sin.copy()
    c.cos_sin[:, :64], c.cos_sin[:, 64:] = 1, 0
    for want, got in zip(c.want(), (dv.kc, dv.vc)):
        np.testing.assert_array_equal(oracle.unpack_rows(got.cpu().numpy()), oracle.unpack_rows(want))


def test_append_special_values():
    """Rows of every size, ties between codes, infinities, NaN, zeros, the largest and the
    smallest scales."""
    r = np.random.default_rng(7)
    c = Append4(7, 200, 2, 2, 128, 16, 13)
    x = values(c.qkv).reshape(200, -1, 128).copy()
    x *= np.float32(2.0) ** r.integers(-30, 30, (200, x.shape[1], 1)).astype(np.float32)
    x[:40] = r.choice([0, 0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -5, -0.25, -2.5], (40,) + x.shape[1:]) * \
        np.float32(2.0) ** r.integers(-20, 14, (40, x.shape[1], 1)).astype(np.float32)
    x[40:44, :, r.integers(0, 128, 9)] = np.inf
    x[44:48, :, r.integers(0, 128, 9)] = -np.inf
    x[48:52, :, r.integers(0, 128, 3)] = np.nan
    x[52:56] = 0
    x[56:58] = -0.0
    x[58] = 3e38
    x[59] = 1e-38
    c.qkv = storage(x.reshape(200, -1), "bf16")
    y = c.qkv.reshape(200, -1, 128)
    c.q, c.k, c.v = y[:, :2], y[:, 2:4], y[:, 4:]
    c.cos_sin = c.cos_sin.copy()
    c.cos_sin[:, :64], c.cos_sin[:, 64:] = 1, 0               # infinities would turn into NaN
    dv = DevAppend(c)
    # without a turn the products with sin = 0 must not meet infinities either: no rotation
    pa.pa_rope_and_cache_fp4(None, None, dv.k, dv.v, dv.kc, dv.vc, dv.slots, None, None, device_errors=dv.errs)
    kc, vc = c.k_cache.copy(), c.v_cache.copy()
    for t, s in enumerate(c.slots):
        kc[s // 16, :, s % 16] = oracle.pack_rows(values(c.k)[t])
        vc[s // 16, :, s % 16] = oracle.pack_rows(values(c.v)[t])
    for want, got in ((kc, dv.kc), (vc, dv.vc)):
        got = got.cpu().numpy()
        np.testing.assert_array_equal(got[..., 64:], want[..., 64:])
        np.testing.assert_array_equal(oracle.unpack_rows(got), oracle.unpack_rows(want))


@pytest.mark.parametrize("hkv,bs,pairs", [(1, 16, 1), (3, 16, 7), (8, 32, 40), (2, 32, 3)])
def test_read_pages(hkv, bs, pairs):
    r = np.random.default_rng(hkv)
    kc, vc = pool(r, 50, hkv, bs), pool(r, 50, hkv, bs)
    kc[..., 64:][r.random(kc[..., 64:].shape) < 0.02] = 0xFF
    p = np.stack([r.permutation(50)[:pairs], r.permutation(60)[:pairs]], 1)
    out = torch.full((2, 60, hkv, bs, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_read_pages_fp4(out[0], out[1], to_dev(kc), to_dev(vc), to_dev(p), device_errors=errs)
    assert pa.pa_read_device_errors(errs) == 0
    for got, c in zip(out, (kc, vc)):
        want = np.full((60, hkv, bs, 128), 7.0)
        want[p[:, 1]] = oracle.unpack_rows(c[p[:, 0]])
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)


def test_buffers_aligned_to_no_more_than_asked():
    c = Append4(21, 45, 8, 2, 128, 16, 5)
    dv = DevAppend(c)
    dv.kc, dv.vc, dv.q_out = (shifted(x, 16) for x in (dv.kc, dv.vc, dv.q_out))
    assert dv.call() == 0
    check_append(c, dv)
    # read back: destinations on 32 bytes, on 16 refused
    pairs = to_dev(np.array([[0, 1], [3, 0]]))
    blank = torch.full((2, 2, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ko, vo = shifted(blank, 32), shifted(blank, 32)
    pa.pa_read_pages_fp4(ko, vo, dv.kc, dv.vc, pairs, device_errors=dv.errs)
    assert pa.pa_read_device_errors(dv.errs) == 0
    for got, pool_ in ((ko, dv.kc), (vo, dv.vc)):
        want = oracle.unpack_rows(pool_.cpu().numpy()[[3, 0]])
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    for outs in ((shifted(blank, 16), vo), (ko, shifted(blank, 16))):
        with pytest.raises(pa.PaError, match="pa_read_pages_fp4"):
            pa.pa_read_pages_fp4(*outs, dv.kc, dv.vc, pairs, device_errors=dv.errs)
    # decode
    c = Decode4(22, [1, 40, 300], 1, 8, 2, 16, spread=3)
    dv = Dev(c)
    dv.q, dv.kc, dv.vc, dv.out = (shifted(x, 16) for x in (dv.q, dv.kc, dv.vc, dv.out))
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


def test_read_all_codes_under_all_scales():
    rows = np.zeros((16, 1, 16, 72), np.uint8)
    rows[..., :64] = np.tile(np.arange(256, dtype=np.uint8).reshape(4, 64), (64, 1)).reshape(16, 1, 16, 64)
    rows[..., 64:] = np.arange(2048).reshape(16, 1, 16, 8) % 0xE3
    out = torch.zeros(2, 16, 1, 16, 128, dtype=torch.bfloat16, device=DEV)
    p = torch.arange(16, device=DEV)[:, None].expand(16, 2).contiguous()
    pa.pa_read_pages_fp4(out[0], out[1], to_dev(rows), to_dev(rows), p)
    np.testing.assert_array_equal(out[0].double().cpu().numpy(), oracle.unpack_rows(rows))


def test_read_bad_pages():
    r = np.random.default_rng(9)
    kc = pool(r, 4, 2, 16)
    p = to_dev(np.array([[0, 1], [-1, 0], [4, 2], [1, 3], [2, -5], [3, 2 ** 40]]))
    out = torch.full((2, 3, 2, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_read_pages_fp4(out[0], out[1], to_dev(kc), to_dev(kc), p, device_errors=errs)
    assert pa.pa_read_device_errors(errs) == pa.PA_DEVERR_BAD_BLOCK
    want = np.full((3, 2, 16, 128), 7.0)
    want[1] = oracle.unpack_rows(kc[0])
    np.testing.assert_array_equal(out[0].double().cpu().numpy(), want)


class Dev:
    def __init__(self, c):
        self.c = c
        self.q = to_dev(c.q if c.q_len > 1 else c.q[:, 0], True)
        self.kc, self.vc = to_dev(c.k_cache), to_dev(c.v_cache)
        self.tables, self.lens = to_dev(c.tables), to_dev(c.lens)
        self.out = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device=DEV)
        self.errs = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(self, out=None, **kw):
        c = self.c
        kw = dict(max_context_len=int(c.lens.max()), window=c.window, sinks=c.sinks, device_errors=self.errs) | kw
        return pa.pa_decode_fp4(self.out if out is None else out, self.q, self.kc, self.vc, self.tables, self.lens,
                                c.scale, c.hkv, **kw)

    def errors(self):
        return pa.pa_read_device_errors(self.errs)


def check(c, got):
    want, parts = c.want()
    got, bar = out_as_f64(got).reshape(want.shape), c.bar(want, parts)
    err = np.abs(got - want)
    assert np.all(err <= bar), f"error {np.nanmax(err / bar):.2f} of its bar, {np.isnan(err).sum()} NaN"


KINDS = [(1, 32, 8, 16), (1, 3, 3, 32), (2, 8, 2, 16), (8, 4, 4, 32), (1, 8, 1, 16), (1, 2, 1, 32)]


@pytest.mark.parametrize("q_len,hq,hkv,bs", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (33, 0), (64, 17), (100, 70), (5000, 2)])
def test_decode_small_calls(q_len, hq, hkv, bs, window, sinks):
    lens = [q_len, q_len + 1, 15 + q_len, 16 + q_len, 33 + q_len, 97, 131, 300]
    c = Decode4(q_len + hq + bs + window, lens, q_len, hq, hkv, bs, window, sinks, spread=3)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("q_len,hq,hkv,bs", [(1, 16, 8, 16), (1, 16, 16, 16), (2, 8, 2, 32), (8, 1, 1, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 4), (90, 33)])
def test_decode_large_calls_in_shares(q_len, hq, hkv, bs, window, sinks):
    r = np.random.default_rng(hq + bs)
    lens = [int(x) for x in r.integers(q_len, 400, 37)] + [6000, q_len, 3000]
    c = Decode4(hq + hkv + bs, lens, q_len, hq, hkv, bs, window, sinks, spread=2)
    dv = Dev(c)
    width = 120000 // bs
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    tables[:, :dv.tables.shape[1]] = dv.tables
    dv.tables = tables
    dv.call(max_context_len=120000)
    assert dv.errors() == 0
    check(c, dv.out)
    again = torch.empty_like(dv.out)
    dv.call(again, max_context_len=120000, workspace=torch.full((64 << 20,), 0x7F, dtype=torch.uint8, device=DEV))
    assert torch.equal(again.view(torch.int16), dv.out.view(torch.int16)), "not the same bits twice"


@pytest.mark.parametrize("q_len,hq,hkv,B,longest", [(1, 32, 8, 12, 900), (2, 32, 8, 30, 300), (1, 8, 8, 190, 150),
                                                    (8, 8, 8, 5, 2000), (1, 4, 4, 3, 3000)])
def test_decode_middling_calls(q_len, hq, hkv, B, longest):
    r = np.random.default_rng(B)
    lens = [int(x) for x in r.integers(q_len, longest, B - 1)] + [longest]
    c = Decode4(B + q_len, lens, q_len, hq, hkv, 16, spread=2)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


def test_decode_empty_sequences_and_bad_pages():
    c = Decode4(40, [0, 40, 0, 90], 1, 4, 2, 16)
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0 and bool((dv.out[[0, 2]] == 0).all())
    check(c, dv.out)
    # a page that is none: its tokens are not seen
    dv.tables[3, 1] = c.nb + 5
    dv.call()
    assert dv.errors() == pa.PA_DEVERR_BAD_BLOCK
    t = [x for x in range(90) if x // 16 != 1]
    k, v = (oracle.unpack_rows(p)[c.tables[3][np.array(t) // 16], :, np.array(t) % 16] for p in (c.k_cache, c.v_cache))
    q = values(c.q)[3, 0].astype(np.float64)
    for i in range(4):
        s = c.scale * (k[:, i // 2] @ q[i])
        w = np.exp(s - s.max())
        w /= w.sum()
        np.testing.assert_allclose(out_as_f64(dv.out)[3, i], w @ v[:, i // 2], atol=0.05)


def test_decode_rows_of_the_largest_and_smallest_scales():
    """Values up to 6 * 10240 and down to 2^-18 enter the products exactly."""
    c = Decode4(41, [200, 65], 1, 8, 2, 16)
    r = np.random.default_rng(41)
    for pool_ in (c.k_cache, c.v_cache):
        keep = pool_[..., 64:] != 0xFF
        pool_[..., 64:] = np.where(keep, r.choice([0x01, 0x05, 0x08, 0x30, 0xE2], pool_[..., 64:].shape), 0xFF)
    c.scale = float(np.float32(2.0 ** -22))
    dv = Dev(c)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


def test_decode_captured_and_replayed_on_two_streams():
    cs = [Decode4(50 + i, [100, 700, 5], 1, 8, 2, 16) for i in range(2)]
    dvs = [Dev(c) for c in cs]
    graphs = []
    for dv in dvs:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            dv.call(workspace=ws)
            with torch.cuda.graph(g, stream=s):
                dv.call(workspace=ws)
        graphs.append((s, g, ws))
    torch.cuda.synchronize()
    for dv in dvs:
        dv.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, g, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, dv in zip(cs, dvs):
        assert dv.errors() == 0
        check(c, dv.out)


@pytest.mark.parametrize("limit", [0, 64])
def test_decode_expired_waits_report_and_leave_the_context_usable(limit):
    c = Decode4(60, [100, 2000, 900] * 20, 1, 8, 2, 16)
    dv = Dev(c)
    try:
        pa.pa_debug_set_wait_limit(limit)
        for _ in range(3):
            dv.call()
        flags = dv.errors()
    finally:
        pa.pa_debug_set_wait_limit(-1)
    assert flags & ~pa.PA_DEVERR_TIMEOUT == 0 and (limit or flags)
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


def test_pools_past_32_bits():
    """Append, read back and decode in the last pages of pools of more than 2^32 bytes."""
    hkv, bs, T = 8, 16, 40
    nb = (1 << 32) // (hkv * bs * 72) + 60
    r = np.random.default_rng(61)
    kc, vc = (torch.empty(nb, hkv, bs, 72, dtype=torch.uint8, device=DEV) for _ in range(2))
    pages = nb - 1 - np.arange(3)
    qkv = torch.from_numpy(r.standard_normal((T, 3 * hkv, 128))).bfloat16().to(DEV)
    q, k, v = qkv.split([hkv, hkv, hkv], 1)
    slots = torch.from_numpy((pages[np.arange(T) // bs] * bs + np.arange(T) % bs).astype(np.int64)).to(DEV)
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rope_and_cache_fp4(None, None, k, v, kc, vc, slots, None, None, device_errors=errs)
    host = [oracle.pack_rows(x.float().cpu().numpy()) for x in (k, v)]
    back = torch.zeros(2, 3, hkv, bs, 128, dtype=torch.bfloat16, device=DEV)
    pairs = torch.from_numpy(np.stack([pages, np.arange(3)], 1).astype(np.int64)).to(DEV)
    pa.pa_read_pages_fp4(back[0], back[1], kc, vc, pairs, device_errors=errs)
    for got, want in zip(back, host):
        rows = got.transpose(1, 2).reshape(-1, hkv, 128)[:T].double().cpu().numpy()
        np.testing.assert_array_equal(rows, oracle.unpack_rows(want))
    out = torch.empty(1, hkv, 128, dtype=torch.bfloat16, device=DEV)
    table = torch.from_numpy(pages.astype(np.int32))[None].to(DEV)
    pa.pa_decode_fp4(out, q[-1:].contiguous(), kc, vc, table, torch.tensor([T], dtype=torch.int32, device=DEV), 128 ** -0.5,
                     hkv, T, device_errors=errs)
    kk, vv = (oracle.unpack_rows(x) for x in host)
    for h in range(hkv):
        s = 128 ** -0.5 * (kk[:, h] @ q[-1, h].double().cpu().numpy())
        w = np.exp(s - s.max())
        w /= w.sum()
        np.testing.assert_allclose(out_as_f64(out)[0, h], w @ vv[:, h], rtol=2.0 ** -8, atol=2.0 ** -11 * 8 * np.abs(vv[:, h]).max())
    assert pa.pa_read_device_errors(errs) == 0


def test_python_refusals():
    c = Decode4(62, [40, 30], 1, 8, 2, 16)
    for name, bad, err in (("kc", None, TypeError), ("q", "float", TypeError), ("tables", "long", TypeError)):
        dv = Dev(c)
        setattr(dv, name, getattr(getattr(dv, name), bad)() if bad else dv.kc.view(torch.int8))
        with pytest.raises(err):
            dv.call()
    dv = Dev(c)
    dv.kc, dv.vc = dv.kc[..., :64].contiguous(), dv.vc[..., :64].contiguous()
    with pytest.raises(ValueError):
        dv.call()
    out = torch.zeros(2, 4, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    dv, pairs = Dev(c), torch.zeros(1, 2, dtype=torch.int64, device=DEV)
    for args, err in (((out[0], out[1].float(), dv.kc, dv.vc, pairs), TypeError),
                      ((out[0], out[1, :3], dv.kc, dv.vc, pairs), ValueError),
                      ((out[0], out[1], dv.kc, dv.vc, pairs.int()), TypeError),
                      ((out[0], out[1], dv.kc, dv.vc, pairs[0]), ValueError),
                      ((out[0, :, :1], out[1, :, :1], dv.kc, dv.vc, pairs), ValueError)):
        with pytest.raises(err):
            pa.pa_read_pages_fp4(*args)
