"""4-bit rows and prompts without a GPU: the oracle pinned to hand-worked rows, to torch and
to the decode oracle, and the host checks of the calls."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
from prefill_cases import Prompts
from rope_cases import values


def test_code_values():
    want = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert oracle.E2M1_VALUES.tolist() == want + [-x for x in want]


def test_scale_values_are_the_halves_with_those_upper_bits():
    halves = torch.from_numpy((np.arange(256, dtype=np.int16) << 7)).view(torch.float16).double().numpy()
    np.testing.assert_array_equal(oracle.SCALE_VALUES, halves)


def test_a_row_worked_out_by_hand():
    x = np.zeros((1, 128), np.float32)
    # amax 6, scale 1 (half 0x3c00: byte 0x78); ties go to the even code
    x[0, :16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 0.26, 4.9, 5.1, -0.74, 3.4, 100e-9]
    x[0, 16:32] = 2.0 ** -30                                  # below half the least scale: zeros
    x[0, 32] = 6.6                                            # amax / 6 = 1.1: 1.125 (0x79); 6.6 / 1.125 = 5.87
    x[0, 48] = 1e30                                           # beyond the largest scale: 6 * 10240
    x[0, 64] = np.inf
    x[0, 80] = np.nan
    x[0, 96] = 6 * 2.0 ** -17                                 # the least scale
    row = oracle.pack_rows(x)[0]
    codes = np.stack([row[:64] & 15, row[:64] >> 4], -1).reshape(-1)
    assert codes[:16].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 14, 1, 6, 7, 9, 5, 0]
    assert row[64:].tolist() == [0x78, 0, 0x79, 0xE2, 0xE2, 0xFF, 0x01, 0]
    assert codes[16:32].tolist() == [0] * 16 and codes[32] == 7 and codes[48] == 7 and codes[64] == 7
    v = oracle.unpack_rows(row)
    assert v[0] == 6 and v[32] == 6.75 and v[48] == 61440 and np.isnan(v[80:96]).all() and v[96] == 6 * 2.0 ** -17


def test_pack_unpack_keeps_what_it_has():
    r = np.random.default_rng(0)
    rows = r.integers(0, 256, (200, 72)).astype(np.uint8)
    rows[:, 64:] = r.integers(8, 0xE2, (200, 8))
    rows[:, :64:8] |= 7                                       # each block's largest is 6 times its scale
    x = oracle.unpack_rows(rows)
    np.testing.assert_array_equal(oracle.unpack_rows(oracle.pack_rows(x.astype(np.float32))), x)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("f32", 4, 2, 64), ("bf16", 8, 1, 128)])
def test_prompt_oracle_is_the_decode_oracle(dtype, hq, hkv, d):
    """New tokens of equal number: decode_multi_f64."""
    c = Prompts(3, dtype, [5, 5, 5], [0, 20, 33], hq, hkv, d, 16)
    out, _ = c.want()
    q = c.q.reshape(3, 5, hq, d)
    want = oracle.decode_multi_f64(q, c.k_cache, c.v_cache, c.tables, c.lens, c.scale, hkv, dtype)
    np.testing.assert_allclose(out.reshape(want.shape), want, atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(0, 0), (7, 0), (7, 3), (1, 5)])
def test_prompt_oracle_equals_dense_attention(window, sinks):
    n, had, d = 19, 12, 64
    c = Prompts(4, "f32", [n], [had], 2, 2, d, 16, window, sinks)
    t = np.arange(n + had)
    k, v = (torch.from_numpy(np.nan_to_num(x[np.where(c.tables[0][t // 16] < c.nb, c.tables[0][t // 16], 0).clip(0), :, t % 16])).double()
            for x in (c.k_cache, c.v_cache))
    p = torch.arange(had, had + n)[:, None]
    see = torch.from_numpy(t) <= p
    if window:
        see &= (p - torch.from_numpy(t) < window) | (torch.from_numpy(t) < sinks)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(c.q).double().transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), attn_mask=see, scale=c.scale)
    np.testing.assert_allclose(c.want()[0], want.transpose(0, 1).numpy(), atol=1e-12)


def _buffer():
    buf = (ctypes.c_uint8 * 4096)()
    return buf, (ctypes.addressof(buf) + 255) & ~255


def _prefill(**over):
    buf, p = _buffer()
    a = dict(out=p, q=p, k=p, v=p, bt=p, cl=p, qs=p, scale=1.0, hkv=8, b=2, t=100, hq=32, d=128, bs=16, nb=64, mbps=8,
             maxlen=100, window=8, sinks=2, dtype=1, ws=p, wsb=1 << 30, errs=None, stream=None)
    a.update(over)
    return pa.library().pa_prefill(*a.values())


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("over,status", [
    (dict(b=0), 0), (dict(t=0), 0), (dict(b=-1), -1), (dict(t=-1), -1), (dict(d=96), -2), (dict(bs=8), -2),
    (dict(hq=30), -1), (dict(hq=24), -2), (dict(hkv=0), -1), (dict(maxlen=129), -1), (dict(maxlen=-1), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(window=0), -1), (dict(dtype=2), -2), (dict(scale=0.0), -1),
    (dict(scale=-1.0), -1), (dict(scale=NAN), -1), (dict(scale=INF), -1), (dict(nb=0), -1), (dict(mbps=-1), -1),
    (dict(out=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(bt=None), -1),
    (dict(cl=None), -1), (dict(qs=None), -1), (dict(nb=2 ** 30), -1), (dict(t=2 ** 30), -1)])
def test_prefill_refusals(over, status):
    assert _prefill(**over) == status


def test_prefill_workspace_size_of_what_is_refused():
    f = pa.pa_prefill_workspace_size
    assert f(-1, 1, 8, 8, 128) == f(1, -1, 8, 8, 128) == f(1, 1, 9, 8, 128) == f(1, 1, 8, 8, 96) == f(1, 1, 8, 0, 64) == 0


def _read(**over):
    buf, p = _buffer()
    a = dict(ko=p, vo=p, k=p, v=p, pairs=p, n=3, hkv=8, d=128, bs=16, ns=10, nd=10, errs=None, stream=None)
    a.update(over)
    return pa.library().pa_read_pages_fp4(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(n=0), 0), (dict(n=-1), -1), (dict(d=64), -2), (dict(bs=64), -2), (dict(hkv=0), -1), (dict(ns=0), -1),
    (dict(nd=0), -1), (dict(ko=None), -1), (dict(vo=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(pairs=None), -1), (dict(hkv=1 << 20), -1)])
def test_read_refusals(over, status):
    assert _read(**over) == status


def test_misaligned_buffers_are_refused():
    buf, p = _buffer()
    for name in ("ko", "vo", "k", "v"):
        assert _read(**{name: p + 8}) == -1
    for name in ("out", "q", "k", "v"):
        assert _prefill(**{name: p + 8}) == -1


@pytest.mark.parametrize("name", ["ko", "vo"])
def test_read_wants_destinations_on_32_bytes(name):
    buf, p = _buffer()
    assert p % 32 == 0
    assert _read(**{name: p + 16}) == -1


def _decode(**over):
    buf, p = _buffer()
    a = dict(out=p, q=p, k=p, v=p, bt=p, cl=p, scale=1.0, hkv=8, b=2, hq=32, ql=1, d=128, bs=16, nb=64, mbps=8,
             maxlen=100, window=8, sinks=2, ws=p, wsb=1 << 30, errs=None, stream=None)
    a.update(over)
    return pa.library().pa_decode_fp4(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(b=0), 0), (dict(d=64), -2), (dict(bs=8), -2), (dict(hq=24), -2), (dict(ql=4), -2), (dict(hkv=0), -1),
    (dict(maxlen=129), -1), (dict(window=0), -1), (dict(out=None), -1), (dict(bt=None), -1), (dict(k=8), -1)])
def test_decode_refusals(over, status):
    assert _decode(**over) == status


def _append(**over):
    buf, p = _buffer()
    a = dict(qo=p, q=p, k=p, v=p, kc=p, vc=p, slots=p, pos=p, cs=p, qs=4096, ks=1024, vs=1024, t=1, hq=32, hkv=8, d=128,
             rot=128, inter=0, most=10, bs=16, nb=4, errs=None, stream=None)
    a.update(over)
    return pa.library().pa_rope_and_cache_fp4(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(t=0), 0), (dict(t=-1), -1), (dict(d=64), -2), (dict(bs=8), -2), (dict(rot=24), -2), (dict(most=0), -1),
    (dict(ks=4), -1), (dict(kc=None), -1), (dict(slots=None), -1), (dict(q=None), -1), (dict(kc=8), -1)])
def test_append_refusals(over, status):
    assert _append(**over) == status


def test_python_refuses_what_does_not_fit():
    z = torch.zeros
    cpu = z(4, 2, 16, 72, dtype=torch.uint8)
    with pytest.raises(ValueError):                           # not CUDA tensors
        pa.pa_read_pages_fp4(z(4, 2, 16, 128, dtype=torch.bfloat16), z(4, 2, 16, 128, dtype=torch.bfloat16), cpu, cpu,
                             z(1, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        pa.pa_prefill(z(3, 2, 64), z(3, 2, 64), z(4, 2, 16, 64), z(4, 2, 16, 64), z(1, 2, dtype=torch.int32),
                      z(1, dtype=torch.int32), z(2, dtype=torch.int32), 1.0, 2, 16)
    with pytest.raises(ValueError):
        pa.pa_prefill(z(3, 2, 64), z(3, 2, 64), z(4, 2, 16, 64), z(4, 2, 16, 64), z(1, 2, dtype=torch.int32),
                      z(1, dtype=torch.int32), z(2, dtype=torch.int32), 1.0, 2, 16, prepare=True)
    with pytest.raises(TypeError):
        pa.pa_read_pages_fp4(None, None, None, None, None)
