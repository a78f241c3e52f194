"""Prompts and 4-bit pools in further calls that their documentation allows: swapped pages, one
graph of a whole step, calls without a plan replayed with other data, the widest tables and the
largest float32 pools, sequences without tokens among ones whose keys are cut."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
from fp4_cases import Decode4
from gpu_helpers import DEV, out_as_f64, to_dev
from prefill_cases import Prompts
from test_gpu_fp4 import Dev as Dev4, check as check4
from test_gpu_prefill import Dev, check

pytestmark = pytest.mark.gpu


def test_pages_of_4_bit_rows_swapped_out_and_in():
    c = Decode4(80, [100, 300, 17], 1, 8, 2, 16)
    dv = Dev4(c)
    host = [torch.zeros(dv.kc.shape, dtype=torch.uint8).pin_memory() for _ in range(2)]
    pages = np.unique(c.tables[(c.tables >= 0) & (c.tables < c.nb)]).astype(np.int64)
    there = np.random.default_rng(80).permutation(c.nb)[:len(pages)]
    out = to_dev(np.stack([pages, there], 1))
    pa.pa_swap_blocks(dv.kc, dv.vc, *host, out, device_errors=dv.errs)
    torch.cuda.synchronize()
    for pool in (dv.kc, dv.vc):
        pool.fill_(0xFF)
    pa.pa_swap_blocks(*host, dv.kc, dv.vc, out.flip(1).contiguous(), device_errors=dv.errs)
    dv.call()
    assert dv.errors() == 0
    check4(c, dv.out)


def test_one_graph_of_append_read_back_attention_and_decode():
    """A step over 4-bit pools in one graph, its buffers' contents new at each replay: the same
    bits as the calls one by one."""
    hq, hkv, bs, T, nb = 8, 2, 16, 70, 12
    r = np.random.default_rng(81)
    s = torch.cuda.Stream()
    order = torch.from_numpy(r.permutation(nb)).to(DEV)
    pages = -(-T // bs)
    pos = torch.arange(T, device=DEV)
    slots = order[pos // bs] * bs + pos % bs
    table = order[:pages][None].int().contiguous()
    pairs = torch.stack([order[:pages], torch.arange(pages, device=DEV)], 1).contiguous()
    here = torch.arange(pages, dtype=torch.int32, device=DEV)[None].contiguous()
    cs = torch.randn(T, 128, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    lens, starts = i32(T), i32(0, T)
    x = torch.randn(T, hq + 2 * hkv, 128, device=DEV).bfloat16()
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(pa.pa_prefill_workspace_size(T, 1, hq, hkv, 128), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(pa.pa_decode_window_workspace_size(1, hq, hkv, 128, bs, T), dtype=torch.uint8, device=DEV)

    def buffers():
        return dict(q=torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV), out=torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV),
                    last=torch.full((1, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV),
                    k=torch.full((nb, hkv, bs, 72), 0xFF, dtype=torch.uint8, device=DEV), v=torch.full((nb, hkv, bs, 72), 0xFF, dtype=torch.uint8, device=DEV),
                    kb=torch.full((pages, hkv, bs, 128), float("nan"), dtype=torch.bfloat16, device=DEV),
                    vb=torch.full((pages, hkv, bs, 128), float("nan"), dtype=torch.bfloat16, device=DEV))

    def step(b):
        pa.pa_rope_and_cache_fp4(b["q"], x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], b["k"], b["v"], slots, pos, cs, device_errors=errs)
        pa.pa_read_pages_fp4(b["kb"], b["vb"], b["k"], b["v"], pairs, device_errors=errs)
        pa.pa_prefill(b["out"], b["q"], b["kb"], b["vb"], here, lens, starts, 128 ** -0.5, hkv, T, workspace=ws, device_errors=errs)
        pa.pa_decode_fp4(b["last"], b["q"][-1:], b["k"], b["v"], table, lens, 128 ** -0.5, hkv, T, workspace=ws2, device_errors=errs)

    inside = buffers()
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(inside)
        with torch.cuda.graph(g, stream=s):
            step(inside)
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(torch.randn_like(x))
        for t in inside.values():
            t.view(torch.uint8).fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        outside = buffers()
        for n in ("k", "v", "kb", "vb"):
            outside[n].view(torch.uint8).fill_(0xFF)
        step(outside)
        for n in inside:
            assert torch.equal(inside[n].view(torch.uint8), outside[n].view(torch.uint8)), n
        # the last token's two attentions: weights in bf16 (2^-8 of each) and in halves (2^-11), their
        # products with V at most its largest element in sum, each result rounded once (2^-8)
        a, b = inside["out"][-1].double(), inside["last"][0].double()
        most = inside["vb"].double().nan_to_num(0).abs().max()
        assert bool(((a - b).abs() <= 2.0 ** -8 * (a.abs() + b.abs()) + (2.0 ** -8 + 2.0 ** -10) * most).all())
    assert pa.pa_read_device_errors(errs) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_without_a_plan_captured_and_replayed(dtype):
    c = Prompts(82, dtype, [20, 1, 33, 7, 60], [100, 0, 17, 300, 0], 4, 2, 128, 16, before=1, behind=2)
    dv = Dev(c)
    most = int(c.lens.max())
    ws = torch.empty(pa.pa_prefill_workspace_size(c.rows, 5, 4, 2, 128), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        dv.call(workspace=ws)
        with torch.cuda.graph(g, stream=s):
            dv.call(workspace=ws)
    torch.cuda.synchronize()
    for cut in (0, 1, 5):
        lens, starts = c.lens.copy(), c.starts.copy()
        lens[4] -= cut                                        # fewer new tokens of the last sequence
        starts[5] -= cut
        dv.lens.copy_(torch.from_numpy(lens))
        dv.starts.copy_(torch.from_numpy(starts))
        dv.q.copy_(dv.q.flip(0))
        dv.out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        again = torch.full_like(dv.out, 7.0)
        dv.call(again, max_context_len=most)
        assert torch.equal(again, dv.out) and dv.errors() == 0
        assert bool((dv.out[int(starts[5]):] == 7.0).all()) and bool((dv.out[:1] == 7.0).all())
        assert not bool(torch.isnan(dv.out).any())


@pytest.mark.parametrize("dtype,new,had", [("bf16", [100], [5000]), ("f32", [40, 3], [0, 700]), ("bf16", [700, 900, 30], [0, 300, 2000])])
def test_tables_of_the_widest_bound(dtype, new, had):
    """A bound of 2^28 tokens, of which the sequences use a few: the host takes another way."""
    c = Prompts(83, dtype, new, had, 8, 4, 64, 16)
    dv = Dev(c)
    wide = torch.full((len(new), 1 << 24), -1, dtype=torch.int32, device=DEV)
    wide[:, :dv.tables.shape[1]] = dv.tables
    dv.tables = wide
    dv.call(max_context_len=1 << 28)
    assert dv.errors() == 0
    check(c, dv.out)


def test_float32_pools_past_32_bits():
    hkv, d, bs = 8, 128, 16
    nb = (1 << 32) // (hkv * bs * d * 4) + 40
    c = Prompts(84, "f32", [50], [200], 16, hkv, d, bs)
    dv = Dev(c)
    pools = []
    for small in (dv.kc, dv.vc):
        big = torch.empty(nb, hkv, bs, d, device=DEV)
        big[nb - c.nb:].copy_(small)
        pools.append(big)
    dv.tables = torch.where((dv.tables >= 0) & (dv.tables < c.nb), dv.tables + (nb - c.nb), -1)
    dv.kc, dv.vc = pools
    dv.call()
    assert dv.errors() == 0
    check(c, dv.out)


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_without_tokens_beside_ones_in_shares(d):
    """Rows that see nothing are items too, of a step that is none: zeros, and the keys of the long
    ones are cut as ever."""
    c = Prompts(85, "bf16", [64, 300, 3, 200], [3000, 0, 7000, 0], 8, 2, d, 16)
    ref = Dev(c)
    ref.call()
    assert ref.errors() == 0
    check(c, ref.out)
    dv = Dev(c)
    dv.lens[1] = 0
    dv.lens[3] = 0
    dv.call()
    assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH
    starts = c.starts
    want = out_as_f64(ref.out)
    got = out_as_f64(dv.out)
    for b in (1, 3):
        assert (got[starts[b]:starts[b + 1]] == 0).all()
    full, parts = c.want()
    bar = c.bar(full, parts)
    for b in (0, 2):
        rows = slice(starts[b], starts[b + 1])
        assert (np.abs(got[rows] - full[rows]) <= bar[rows]).all()
