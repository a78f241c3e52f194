"""The operators together, as a serving loop uses them: prompts appended with their
rotation, decode steps through windowed and full layers, a fork with copy-on-write, drafted
tokens verified and in part taken back -- over bf16 pools and over e4m3 pools with page
scales.  What the pools hold is followed by the oracle; every attention output is checked
against 64 bits over that."""
import pathlib
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
import rope_cases
from gpu_helpers import DEV, out_as_f64, storage_to_host, to_dev

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, NB, MOST = 8, 2, 128, 16, 64, 256


class Loop:
    def __init__(self, fp8):
        self.fp8 = fp8
        self.r = np.random.default_rng(20)
        self.bm = pa.BlockManager(NB, BS, initial_free_order=self.r.permutation(NB))
        self.table = rope_cases.table(MOST, D)
        self.d_table = to_dev(self.table)
        shape = (NB, HKV, BS, D)
        if fp8:
            self.host = [np.full(shape, 0x7F, np.uint8) for _ in range(2)]
            self.host_scales = [np.full((NB, HKV), np.nan, np.float32) for _ in range(2)]
            self.scales = [to_dev(s) for s in self.host_scales]
        else:
            self.host = [np.full(shape, 0x7FC0, np.uint16) for _ in range(2)]
        self.pools = [to_dev(x, not fp8) for x in self.host]
        self.errs = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(pa.pa_decode_window_workspace_size(8, 2 * HQ, HKV, D, BS, MOST, 0, 0),
                              dtype=torch.uint8, device=DEV)

    def copy(self, pairs):
        """Copy-on-write: pages, and their scales."""
        if not len(pairs):
            return
        dev = to_dev(pairs)
        pa.pa_copy_blocks(*self.pools, dev, device_errors=self.errs)
        oracle.copy_blocks(*self.host, pairs)
        if self.fp8:
            pa.pa_copy_scales(*self.scales, *self.scales, dev, device_errors=self.errs)
            for s in self.host_scales:
                for a, b in pairs:
                    s[b] = s[a]

    def append(self, slots, positions):
        """Rows of these tokens: returns their rotated q (device) as [T, HQ, D]."""
        T = len(slots)
        qkv = rope_cases.storage(self.r.standard_normal((T, (HQ + 2 * HKV) * D)), "bf16")
        x = qkv.reshape(T, -1, D)
        dev = to_dev(qkv, True)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in dev.split([HQ * D, HKV * D, HKV * D], 1))
        q_out = torch.empty(T, HQ, D, dtype=torch.bfloat16, device=DEV)
        slots, positions = np.asarray(slots, np.int64), np.asarray(positions, np.int64)
        args = (q_out, q, k, v, *self.pools, to_dev(slots), to_dev(positions), self.d_table)
        if self.fp8:
            pa.pa_rope_and_cache_fp8_block(*args, *self.scales, device_errors=self.errs)
        else:
            pa.pa_rope_and_cache(*args, device_errors=self.errs)
        k32 = oracle.rotate_f32(rope_cases.values(x[:, HQ:HQ + HKV]), self.table[positions])
        v_rows = x[:, HQ + HKV:]
        if self.fp8:
            oracle.page_scale_append(k32, slots, self.host[0], self.host_scales[0])
            oracle.page_scale_append(rope_cases.values(v_rows), slots, self.host[1], self.host_scales[1])
        else:
            self.host[0][slots // BS, :, slots % BS] = rope_cases.storage(k32, "bf16")
            self.host[1][slots // BS, :, slots % BS] = v_rows
        return q_out

    def attend(self, ids, q, q_len, window, sinks, lens=None):
        """q [B * q_len, HQ, D] against the sequences' contexts; checked."""
        tables, held = self.bm.build_block_tables(ids, MOST // BS)
        lens = held if lens is None else np.asarray(lens, np.int32)
        q = q.view(len(ids), q_len, HQ, D)
        out = torch.full_like(q, float("nan"))
        args = (out, q, *self.pools, to_dev(tables), to_dev(lens), D ** -0.5)
        kw = dict(window=window, sinks=sinks, workspace=self.ws, device_errors=self.errs)
        if self.fp8:
            pa.pa_decode_fp8_block(*args, *self.scales, HKV, MOST, **kw)
            k, v = (oracle.E4M3_VALUES[c] * s[:, :, None, None].astype(np.float64)
                    for c, s in zip(self.host, self.host_scales))
        else:
            pa.pa_decode_window(*args, HKV, MOST, **kw)
            k, v = (rope_cases.values(c).astype(np.float64) for c in self.host)
        qh = rope_cases.values(storage_to_host(q, "bf16")).astype(np.float64)
        want, parts = oracle.decode_window_f64(qh, k, v, tables, lens, D ** -0.5, window, sinks)
        # half a step of 2^-8 for the weights and for the result, the scores' float32
        bar = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 * 1.01 + 2.0 ** -14 * parts["dots"][..., None] + 2.0 ** -20) * parts["mag"] + 1e-9
        assert np.all(np.abs(out_as_f64(out) - want) <= bar)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_serving_loop(fp8):
    loop, bm = Loop(fp8), None
    bm = loop.bm
    # prompts, in one call
    prompts = {1: 70, 2: 1, 3: 33}
    slots, pos = [], []
    for s, n in prompts.items():
        bm.add_seq(s)
        for p in range(n):
            slots.append(bm.append_slot(s)[0])
            pos.append(p)
    loop.append(slots, pos)
    ids = list(prompts)
    # decode steps; a fork in between, whose last page is shared until one of them writes
    for step in range(20):
        if step == 7:
            bm.fork(1, 9)
            ids.append(9)
        lens = [bm.block_table(s)[1] for s in ids]
        new, cow = bm.append_slots(ids)
        loop.copy(cow)
        assert (len(cow) > 0) == (step == 7)
        q = loop.append(new, lens)
        loop.attend(ids, q, 1, 0, 0)
        loop.attend(ids, q, 1, 24, 3)
    # three drafted tokens beside the next one, verified; the last two are taken back and
    # their slots written again by the tokens that follow
    tables, lens = bm.build_block_tables(ids, MOST // BS)
    slots = [[bm.append_slot(s) for _ in range(4)] for s in ids]
    loop.copy(np.array([(a, b) for s in slots for _, a, b in s if a >= 0], np.int64).reshape(-1, 2))
    flat = [t[0] for s in slots for t in s]
    # (q_len 2 twice: 2 tokens x group 4 = 8 rows)
    first = [s for i, s in enumerate(flat) if i % 4 < 2]
    q = loop.append(first, [n + j for n in lens for j in range(2)])
    loop.attend(ids, q, 2, 24, 3, lens + 2)
    loop.attend(ids, q, 2, 0, 0, lens + 2)
    q = loop.append([s for i, s in enumerate(flat) if i % 4 in (1, 2)], [n + 1 + j for n in lens for j in range(2)])
    loop.attend(ids, q, 2, 5, 0, lens + 3)
    loop.attend(ids, q, 2, 0, 0, lens + 3)
    assert pa.pa_read_device_errors(loop.errs) == 0
    kinds = "fp8" if fp8 else "bf16"
    for dev, host in zip(loop.pools, loop.host):
        got = storage_to_host(dev, kinds)
        same = got == host
        assert np.all(same | (((host & 0x7F) == 0x7F) if fp8 else (host == 0x7FC0)))
    if fp8:
        for dev, host in zip(loop.scales, loop.host_scales):
            np.testing.assert_array_equal(storage_to_host(dev, "f32"), host)


def test_a_captured_step_with_padding():
    """A decode step captured for a padded batch: append, windowed and full attention;
    replayed on other tokens, the padding's rows are left as they were."""
    loop = Loop(True)
    B, live = 4, 3
    for s in range(live):
        loop.bm.add_seq(s)
    slots, pos = [], []
    for s, n in zip(range(live), (40, 17, 3)):
        for p in range(n):
            slots.append(loop.bm.append_slot(s)[0])
            pos.append(p)
    loop.append(slots, pos)
    qkv = torch.zeros(B, (HQ + 2 * HKV) * D, dtype=torch.bfloat16, device=DEV)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    d_slots = torch.full((B,), -1, dtype=torch.int64, device=DEV)
    d_pos = torch.full((B,), -1, dtype=torch.int64, device=DEV)
    tables = torch.full((B, MOST // BS), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    q_out = torch.full((B, HQ, D), 5.0, dtype=torch.bfloat16, device=DEV)
    outs = [torch.empty_like(q_out) for _ in range(2)]

    def step():
        pa.pa_rope_and_cache_fp8_block(q_out, q, k, v, *loop.pools, d_slots, d_pos, loop.d_table, *loop.scales,
                                       device_errors=loop.errs)
        for out, window in zip(outs, (0, 20)):
            pa.pa_decode_fp8_block(out, q_out, *loop.pools, tables, lens, D ** -0.5, *loop.scales, HKV, MOST,
                                   window=window, sinks=2 if window else 0, workspace=loop.ws, device_errors=loop.errs)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(3):
        new, cow = loop.bm.append_slots(list(range(live)))
        assert len(cow) == 0
        t, n = loop.bm.build_block_tables(list(range(live)), MOST // BS)
        x = rope_cases.storage(loop.r.standard_normal((live, (HQ + 2 * HKV) * D)), "bf16")
        qkv[:live] = to_dev(x, True)
        d_slots[:live], d_pos[:live] = to_dev(new), to_dev(n.astype(np.int64) - 1)
        tables[:live], lens[:live] = to_dev(t), to_dev(n)
        graph.replay()
        k32 = oracle.rotate_f32(rope_cases.values(x.reshape(live, -1, D)[:, HQ:HQ + HKV]), loop.table[n - 1])
        oracle.page_scale_append(k32, new, loop.host[0], loop.host_scales[0])
        oracle.page_scale_append(rope_cases.values(x.reshape(live, -1, D)[:, HQ + HKV:]), new, loop.host[1], loop.host_scales[1])
        got = [o.clone() for o in outs]
        assert bool((q_out[live:] == 5.0).all()) and all(bool((o[live:] == 0).all()) for o in got)
        for window, o in zip((0, 20), got):
            eager = torch.empty_like(o)
            pa.pa_decode_fp8_block(eager, q_out, *loop.pools, tables, lens, D ** -0.5, *loop.scales, HKV, MOST,
                                   window=window, sinks=2 if window else 0, device_errors=loop.errs)
            assert torch.equal(eager.view(torch.int16), o.view(torch.int16))
            loop.attend(list(range(live)), q_out[:live].clone(), 1, window, 2 if window else 0)
    assert pa.pa_read_device_errors(loop.errs) == 0


FIRST_CALL = """
import torch
import paged_kv_cache_190_gb300 as pa
g = torch.Generator(device="cuda").manual_seed(0)
q = torch.randn(4, 8, 128, device="cuda", generator=g).bfloat16()
codes = torch.randint(0, 120, (8, 2, 16, 128), device="cuda", generator=g, dtype=torch.uint8)
scales = torch.full((8, 2), 2.0 ** -6, device="cuda")
tables = torch.arange(8, device="cuda", dtype=torch.int32).view(4, 2)
lens = torch.tensor([32, 1, 17, 16], device="cuda", dtype=torch.int32)
ws = torch.empty(1 << 25, device="cuda", dtype=torch.uint8)
out, again = torch.zeros_like(q), torch.zeros_like(q)
call = lambda o: pa.pa_decode_fp8_block(o, q, codes, codes, tables, lens, 0.1, scales, scales, 2, 32, workspace=ws)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call(out)
graph.replay()
call(again)
torch.cuda.synchronize()
assert out.abs().sum() > 0 and torch.equal(out, again)
"""


def test_the_first_call_of_a_process_may_be_captured():
    root = pathlib.Path(__file__).resolve().parent.parent
    done = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


@pytest.mark.parametrize("fp8", [False, True])
def test_the_pools_hold_what_was_written_and_nothing_else(fp8):
    """Prompts, a fork, copy-on-write and decode steps, then every byte of the pools: slots
    that nothing was written to are as they were."""
    loop = Loop(fp8)
    bm = loop.bm
    slots, pos = [], []
    for s, n in {1: 70, 2: 1, 3: 33}.items():
        bm.add_seq(s)
        for p in range(n):
            slots.append(bm.append_slot(s)[0])
            pos.append(p)
    loop.append(slots, pos)
    bm.fork(1, 9)
    ids = [1, 2, 3, 9]
    for _ in range(20):
        lens = [bm.block_table(s)[1] for s in ids]
        new, cow = bm.append_slots(ids)
        loop.copy(cow)
        loop.attend(ids, loop.append(new, lens), 1, 24, 3)
    assert pa.pa_read_device_errors(loop.errs) == 0
    for dev, host in zip(loop.pools, loop.host):
        got = storage_to_host(dev, "fp8" if fp8 else "bf16")
        nan = (host & 0x7F) == 0x7F if fp8 else np.zeros(host.shape, bool)     # a NaN code's sign is free
        np.testing.assert_array_equal(got[~nan], host[~nan])
        assert np.all((got[nan] & 0x7F) == 0x7F)
        assert np.any(host == (0x7F if fp8 else 0x7FC0))
    if fp8:
        for dev, host in zip(loop.scales, loop.host_scales):
            np.testing.assert_array_equal(storage_to_host(dev, "f32"), host)


class NoTruth:
    def __bool__(self):
        raise ArithmeticError("neither")


@pytest.mark.parametrize("fp8", [False, True])
def test_an_argument_without_a_truth_value_raises_its_own_error(fp8):
    loop = Loop(fp8)
    x = torch.zeros(1, HKV, D, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(1, HQ, D, dtype=torch.bfloat16, device=DEV)
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    tables, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    scales = loop.scales if fp8 else ()
    append = pa.pa_rope_and_cache_fp8_block if fp8 else pa.pa_rope_and_cache
    decode = pa.pa_decode_fp8_block if fp8 else pa.pa_decode_window
    for kw in (dict(prepare=NoTruth()), dict(interleaved=NoTruth())):
        with pytest.raises(ArithmeticError):
            append(None, None, x, x, *loop.pools, slots, None, None, *scales, **kw)
    with pytest.raises(ArithmeticError):
        decode(torch.empty_like(q), q, *loop.pools, tables, lens, 1.0, *scales, HKV, BS, window=4, workspace=loop.ws,
               prepare=NoTruth())
