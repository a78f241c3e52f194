"""Codes of 4-bit rows bit by bit: the sign of zeros."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
from gpu_helpers import DEV, to_dev
from rope_cases import storage, values

pytestmark = pytest.mark.gpu


def _stored(x):
    """bf16 rows [T, H, 128] as the append stores them, unrotated: uint8 [2, T, H, 72] of K and V."""
    T, H = x.shape[:2]
    d = to_dev(storage(x, "bf16"), True)
    pools = [torch.full((-(-T // 16), H, 16, 72), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2)]
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rope_and_cache_fp4(None, None, d, d, *pools, torch.arange(T, device=DEV), None, None, device_errors=errs)
    assert pa.pa_read_device_errors(errs) == 0
    return np.stack([p.transpose(1, 2).reshape(-1, H, 72)[:T].cpu().numpy() for p in pools])


@pytest.mark.parametrize("tokens,heads", [(5, 1), (40, 3), (1100, 8)])
def test_codes_byte_for_byte(tokens, heads):
    """Rows of every size: groups whose scale is 0, elements that round to 0 under a larger
    scale, zeros of both signs."""
    r = np.random.default_rng(tokens)
    x = r.standard_normal((tokens, heads, 128)).astype(np.float32)
    x *= np.float32(2.0) ** r.integers(-26, 16, (tokens, heads, 8)).repeat(16, -1).astype(np.float32)
    x[..., 5::16] *= np.float32(2.0 ** -9)
    x[..., 7::32] = 0.0
    x[..., 23::32] = -0.0
    x[0, 0, :16] = -2.0 ** -30                              # (a scale of 0 in the smallest case too)
    x = values(storage(x, "bf16"))
    want = oracle.pack_rows(x)
    assert (want[..., 64:] == 0).any() and (want[..., 64:] > 8).any()
    for got in _stored(x):
        np.testing.assert_array_equal(got, want)


def test_a_scale_of_0_stores_zeros_without_a_sign():
    x = np.full((2, 1, 128), -2.0 ** -30, np.float32)
    x[1, 0, ::2] = -0.0
    for got in _stored(x):
        assert (got == 0).all()


def test_zeros_and_elements_that_round_to_zero():
    """A zero of either sign is code 0; a negative element that rounds to zero keeps its sign."""
    x = np.zeros((1, 1, 128), np.float32)
    x[..., ::16] = 6.0
    x[..., 1::16] = -0.0
    x[..., 2::16] = -2.0 ** -20
    for got in _stored(x):
        codes = np.stack([got[0, 0, :64] & 15, got[0, 0, :64] >> 4], -1).reshape(8, 16)
        assert (codes == [7, 0, 8] + [0] * 13).all()
