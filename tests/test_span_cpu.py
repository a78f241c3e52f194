"""The windowed and the page-scaled decode without a GPU: the oracle pinned to the decode
oracle and to closed forms, and the host checks."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa


def _dense(seed, B, L, hkv, group, d, bs, q_len=1):
    r = np.random.default_rng(seed)
    nb = B * -(-L // bs)
    tables = r.permutation(nb).reshape(B, -1).astype(np.int32)
    return (r.standard_normal((B, q_len, hkv * group, d)), r.standard_normal((nb, hkv, bs, d)),
            r.standard_normal((nb, hkv, bs, d)), tables)


def test_no_window_is_the_decode_oracle():
    q, k, v, t = _dense(0, 3, 50, 2, 2, 64, 16, q_len=2)
    q, k, v = (x.astype(np.float32) for x in (q, k, v))
    lens = np.array([50, 17, 2], np.int32)
    want = oracle.decode_multi_f64(q, k, v, t, lens, 0.125, 2, "f32")
    for window, sinks in ((0, 0), (50, 0), (10 ** 6, 3)):
        got, _ = oracle.decode_window_f64(*(x.astype(np.float64) for x in (q, k, v)), t, lens, 0.125, window, sinks)
        np.testing.assert_allclose(got, want, atol=1e-12)


def test_window_and_sinks_are_a_cut_out_context():
    q, k, v, t = _dense(1, 1, 64, 1, 1, 8, 16)
    got, _ = oracle.decode_window_f64(q, k, v, t, [64], 0.3, window=5, sinks=3)
    pos = [0, 1, 2, 59, 60, 61, 62, 63]
    kk, vv = (np.stack([x[t[0, p // 16], 0, p % 16] for p in pos]) for x in (k, v))
    w = np.exp(0.3 * kk @ q[0, 0, 0])
    np.testing.assert_allclose(got[0, 0, 0], w @ vv / w.sum(), atol=1e-12)
    one, _ = oracle.decode_window_f64(q, k, v, t, [64], 0.3, window=1)
    np.testing.assert_allclose(one[0, 0, 0], v[t[0, 3], 0, 15], atol=1e-12)


def _call(fn="pa_decode_window", **over):
    lib = pa.library()
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 255) & ~255
    a = dict(out=p, q=p, k=p, v=p, bt=p, cl=p, scale=1.0, s0=p, s1=p, hkv=8, b=2, hq=32, ql=1, d=128, bs=16, nb=64,
             mbps=8, maxlen=100, window=8, sinks=2, dtype=1, ws=p, wsb=1 << 30, errs=None, stream=None)
    a.update(over)
    names = ["out", "q", "k", "v", "bt", "cl", "scale"]
    names += ["s0", "s1"] if fn == "pa_decode_fp8_block" else []
    names += ["hkv", "b", "hq", "ql", "d", "bs", "nb", "mbps", "maxlen", "window", "sinks"]
    names += ["dtype"] if fn == "pa_decode_window" else []
    return getattr(lib, fn)(*[a[n] for n in names + ["ws", "wsb", "errs", "stream"]])


@pytest.mark.parametrize("fn", ["pa_decode_window", "pa_decode_fp8_block"])
@pytest.mark.parametrize("over,status", [
    (dict(b=0), 0), (dict(b=-1), -1), (dict(d=96), -2), (dict(bs=8), -2), (dict(hq=30), -1), (dict(hq=24), -2),
    (dict(ql=4), -2), (dict(ql=0), -1), (dict(hkv=0), -1), (dict(maxlen=8 * 16 + 1), -1), (dict(maxlen=-1), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(window=0), -1), (dict(out=None), -1), (dict(bt=None), -1),
    (dict(q=12345), -1), (dict(nb=0), -1), (dict(nb=2 ** 30), -1), (dict(mbps=2 ** 27, maxlen=2 ** 30), -1),
])
def test_host_checks(fn, over, status):
    assert _call(fn, **over) == status


def test_host_checks_of_one_kind_alone():
    assert _call(dtype=5) == -2
    assert _call("pa_decode_fp8_block", d=64) == -2
    assert _call("pa_decode_fp8_block", s0=None) == -1
    assert _call("pa_decode_fp8_block", s1=None) == -1
    size = pa.library().pa_decode_window_workspace_size
    assert size(4, 24, 8, 96, 16, 100, 0, 0) == 0 and size(4, 30, 8, 128, 16, 100, 0, 0) == 0
    assert size(4, 128, 8, 128, 16, 100, 0, 0) == 0 and size(4, 32, 8, 128, 16, 100, -1, 0) == 0


def test_python_calls_refuse_host_tensors():
    q = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    kc = torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16)
    t = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_decode_window(q, q, kc, kc, t, t[0], 1.0, 2, 1, 4)


def test_a_prepared_call_needs_a_workspace():
    q, t = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    pool, codes = torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(8, 2, 16, 128, dtype=torch.uint8)
    lens, scales = torch.ones(2, dtype=torch.int32), torch.ones(8, 2)
    with pytest.raises(ValueError, match="workspace"):
        pa.pa_decode_window(q.clone(), q, pool, pool, t, lens, 1.0, 2, 64, 8, prepare=True)
    with pytest.raises(ValueError, match="workspace"):
        pa.pa_decode_fp8_block(q.clone(), q, codes, codes, t, lens, 1.0, scales, scales, 2, 64, prepare=True)
