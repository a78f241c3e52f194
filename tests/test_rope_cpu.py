"""The rotating appends without a GPU: the oracle pinned to closed forms, the host
checks of the C calls and the argument checks of the Python ones."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
import rope_cases


# ------------------------------------------------------------------- the oracle
def test_rotation_is_a_complex_product():
    r = np.random.default_rng(0)
    x = r.standard_normal((5, 3, 64))
    rows = rope_cases.table(40, 32)[[0, 1, 7, 20, 39]].astype(np.float64)
    z = rows[:, None, :16] + 1j * rows[:, None, 16:]
    got = oracle.rotate_f64(x, rows)
    w = (x[..., :16] + 1j * x[..., 16:32]) * z
    np.testing.assert_allclose(got[..., :32], np.concatenate([w.real, w.imag], -1), atol=1e-15)
    np.testing.assert_array_equal(got[..., 32:], x[..., 32:])
    got = oracle.rotate_f64(x, rows, interleaved=True)
    w = (x[..., 0:32:2] + 1j * x[..., 1:32:2]) * z
    np.testing.assert_allclose(got[..., 0:32:2], w.real, atol=1e-15)
    np.testing.assert_allclose(got[..., 1:32:2], w.imag, atol=1e-15)


def test_rotation_depends_on_the_distance_only():
    r = np.random.default_rng(1)
    q, k = r.standard_normal((1, 1, 64)), r.standard_normal((1, 1, 64))
    t = rope_cases.table(60, 64).astype(np.float64)
    for inter in (False, True):
        dots = [np.sum(oracle.rotate_f64(q, t[[p + 5]], inter) * oracle.rotate_f64(k, t[[p]], inter))
                for p in (0, 11, 50)]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-5)     # the table is float32


@pytest.mark.parametrize("amax,want", [(0.0, 2.0 ** -100), (448.0, 1.0), (448.1, 2.0), (224.0, 0.5),
                                       (1.0, 2.0 ** -8), (0.875, 2.0 ** -9), (0.8751, 2.0 ** -8),
                                       (3e38, 2.0 ** 120)])
def test_power_of_two_scale(amax, want):
    assert oracle.power_of_two_scale(amax) == want


def test_page_scale_append_follows_its_statement():
    codes = oracle.e4m3_encode(np.full((2, 1, 16, 4), 1.0, np.float32))
    scales = np.full((2, 1), 2.0, np.float32)                     # every row stands for 2.0
    x = np.full((3, 1, 4), 3.0, np.float32)
    # page 0 goes on (slots 5, 6), page 1 begins anew (its first slot)
    oracle.page_scale_append(x, [5, 6, 16], codes, scales)
    assert scales[0, 0] == 2.0                                    # 3 / 448 needs less: the scale stays
    v = oracle.E4M3_VALUES[codes]
    assert np.all(v[0, 0, [5, 6]] * 2.0 == 3.0) and np.all(v[0, 0, [0, 15]] * 2.0 == 2.0)
    assert scales[1, 0] == 2.0 ** -7                              # 3 <= 448 2^-7 = 3.5
    assert np.all(v[1, 0, 0] * scales[1, 0] == 3.0)
    big = np.full((1, 1, 4), 4096.0, np.float32)
    oracle.page_scale_append(big, [7], codes, scales)             # 4096 <= 448 * 16
    assert scales[0, 0] == 16.0
    v = oracle.E4M3_VALUES[codes]
    assert np.all(v[0, 0, 7] * 16.0 == 4096.0) and np.all(v[0, 0, [0, 15]] * 16.0 == 2.0)
    assert np.all(v[0, 0, [5, 6]] * 16.0 == 3.0)


# --------------------------------------------------------------------- C checks
def _call(fn="pa_rope_and_cache", **over):
    lib = pa.library()
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 255) & ~255
    a = dict(q_out=p, q=p, k=p, v=p, kc=p, vc=p, slots=p, pos=p, table=p, s0=p, s1=p, qs=4096,
             ks=1024, vs=1024, t=2, hq=32, hkv=8, d=128, rot=128, inter=0, most=64, bs=16, nb=4,
             dtype=1, errs=None, stream=None)
    a.update(over)
    names = ["q_out", "q", "k", "v", "kc", "vc", "slots", "pos", "table"]
    if fn != "pa_rope_and_cache":
        names += ["s0", "s1"]
    names += ["qs", "ks", "vs", "t", "hq", "hkv", "d", "rot", "inter", "most", "bs", "nb"]
    if fn == "pa_rope_and_cache":
        names.append("dtype")
    return getattr(lib, fn)(*[a[n] for n in names + ["errs", "stream"]])


ALL = ["pa_rope_and_cache", "pa_rope_and_cache_fp8", "pa_rope_and_cache_fp8_block"]


@pytest.mark.parametrize("fn", ALL)
@pytest.mark.parametrize("over,status", [
    (dict(t=0), 0), (dict(t=-1), -1), (dict(t=2 ** 26), -1), (dict(hkv=0), -1), (dict(hq=-1), -1), (dict(nb=0), -1),
    (dict(d=96), -2), (dict(bs=8), -2), (dict(rot=24), -2), (dict(rot=144), -2), (dict(rot=-16), -2),
    (dict(rot=0), -1),                              # q without a rotation
    (dict(most=0), -1), (dict(q=None), -1), (dict(q_out=None), -1), (dict(k=None), -1),
    (dict(vc=None), -1), (dict(slots=None), -1), (dict(pos=None), -1), (dict(table=None), -1),
    (dict(qs=4100), -1), (dict(ks=1028), -1), (dict(vs=-1024), -1), (dict(k=12344), -1),
])
def test_host_checks(fn, over, status):
    assert _call(fn, **over) == status


def test_host_checks_of_one_type_alone():
    assert _call(dtype=7) == -2
    for fn in ALL[1:]:
        assert _call(fn, d=64) == -2
        assert _call(fn, s0=None) == -1
        assert _call(fn, s1=None) == -1


def test_copy_scales_host_checks():
    lib = pa.library()
    buf = (ctypes.c_uint8 * 1024)()
    p = (ctypes.addressof(buf) + 255) & ~255
    assert lib.pa_copy_scales(p, p, p, p, p, 0, 8, 4, 4, None, None) == 0
    assert lib.pa_copy_scales(p, p, p, p, p, -1, 8, 4, 4, None, None) == -1
    assert lib.pa_copy_scales(p, p, p, p, p, 1, 0, 4, 4, None, None) == -1
    assert lib.pa_copy_scales(p, p, p, p, p, 1, 8, 0, 4, None, None) == -1
    assert lib.pa_copy_scales(p, p, None, p, p, 1, 8, 4, 4, None, None) == -1


def test_python_calls_refuse_host_tensors():
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    kc = torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        pa.pa_rope_and_cache(x, x, x, x, kc, kc, one, one, torch.zeros(4, 128))
    with pytest.raises(ValueError):
        pa.pa_copy_scales(torch.zeros(2, 2), torch.zeros(2, 2), torch.zeros(2, 2),
                          torch.zeros(2, 2), torch.zeros(1, 2, dtype=torch.int64))
