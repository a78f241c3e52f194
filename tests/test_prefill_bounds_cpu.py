"""Bounds that the host checks of the prompts and the 4-bit pools draw, without a GPU."""
import pytest

from test_fp4_cpu import _prefill, _read


@pytest.mark.parametrize("over", [dict(hkv=65536, bs=32), dict(hkv=1 << 17, bs=16), dict(hkv=131071, bs=16),
                                  dict(hkv=2 ** 31 - 1, bs=16)])
def test_pages_of_more_rows_than_a_grid_holds_are_bad_arguments(over):
    assert _read(**over) == -1
    assert _read(n=0, **over) == -1


@pytest.mark.parametrize("over", [dict(hkv=65535, bs=32), dict(hkv=65536, bs=16), dict(hkv=131070, bs=16)])
def test_the_largest_pages_are_good_arguments(over):
    assert _read(n=0, **over) == 0


@pytest.mark.parametrize("scale,status", [(2.3e38, 0), (1e-45, 0), (2.4e38, -1), (3.4e38, -1)])
def test_a_scale_whose_base_2_form_overflows_is_a_bad_argument(scale, status):
    assert _prefill(scale=scale, b=0) == status
