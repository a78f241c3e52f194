"""The prompt attention on the GPU against the oracle; prefill_cases.Prompts.bar has the
error bars."""
import numpy as np
import pytest
import torch

import paged_kv_cache_190_gb300 as pa
from gpu_helpers import DEV, out_as_f64, to_dev
from prefill_cases import Prompts

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
