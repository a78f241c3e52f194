"""Prompts and decode steps together, as a serving loop uses them: prompts filled in chunk by
chunk (append, then attention of the chunk over what the cache holds), decoded from then on
-- over bf16 pools, and over 4-bit pools whose pages are read back for the prompts'
attention.  What the pools hold is followed by the oracle; every attention output is checked
against 64 bits over that."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_190_gb300 as pa
import rope_cases
from gpu_helpers import DEV, out_as_f64, storage_to_host, to_dev

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, NB, MOST = 8, 2, 128, 16, 80, 512


class Loop:
    def __init__(self, fp4):
        self.fp4 = fp4
        self.r = np.random.default_rng(30)
        self.bm = pa.BlockManager(NB, BS, initial_free_order=self.r.permutation(NB))
        self.table = rope_cases.table(MOST, D)
        self.d_table = to_dev(self.table)
        if fp4:
            self.host = [np.full((NB, HKV, BS, 72), 0xFF, np.uint8) for _ in range(2)]
            self.scratch = torch.full((2, NB, HKV, BS, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        else:
            self.host = [np.full((NB, HKV, BS, D), 0x7FC0, np.uint16) for _ in range(2)]
        self.pools = [to_dev(x, not fp4) for x in self.host]
        self.errs = torch.zeros(1, dtype=torch.int32, device=DEV)

    def append(self, slots, positions):
        T = len(slots)
        qkv = rope_cases.storage(self.r.standard_normal((T, (HQ + 2 * HKV) * D)), "bf16")
        x = qkv.reshape(T, -1, D)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in to_dev(qkv, True).split([HQ * D, HKV * D, HKV * D], 1))
        q_out = torch.empty(T, HQ, D, dtype=torch.bfloat16, device=DEV)
        slots, positions = np.asarray(slots, np.int64), np.asarray(positions, np.int64)
        call = pa.pa_rope_and_cache_fp4 if self.fp4 else pa.pa_rope_and_cache
        call(q_out, q, k, v, *self.pools, to_dev(slots), to_dev(positions), self.d_table, device_errors=self.errs)
        k32 = oracle.rotate_f32(rope_cases.values(x[:, HQ:HQ + HKV]), self.table[positions])
        v_rows = x[:, HQ + HKV:]
        rows = (oracle.pack_rows(k32), oracle.pack_rows(rope_cases.values(v_rows))) if self.fp4 else \
            (rope_cases.storage(k32, "bf16"), v_rows)
        for host, new in zip(self.host, rows):
            host[slots // BS, :, slots % BS] = new
        return q_out

    def held(self):
        if self.fp4:
            return [oracle.unpack_rows(x) for x in self.host]
        return [rope_cases.values(x).astype(np.float64) for x in self.host]

    def check(self, out, want, parts, half):
        bar = 2.0 ** -8 * np.abs(want) + (half * 1.01 + 2.0 ** -13 * parts["dots"][..., None] + 2.0 ** -12) * parts["mag"] + 1e-9
        err = np.abs(out_as_f64(out) - want)
        assert np.all(err <= bar), f"error {np.nanmax(err / bar):.2f} of its bar"

    def prompts(self, ids, new, q, window, sinks):
        """The new tokens' attention: over the pools, or over their pages read back."""
        tables, lens = self.bm.build_block_tables(ids, MOST // BS)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        out = torch.full_like(q, float("nan"))
        pools, d_tables = self.pools, tables
        if self.fp4:
            pages = np.concatenate([t[:-(-int(n) // BS)] for t, n in zip(tables, lens)])
            d_tables = np.full_like(tables, -1)
            at = 0
            for b, n in enumerate(lens):
                m = -(-int(n) // BS)
                d_tables[b, :m] = at + np.arange(m)
                at += m
            pairs = np.stack([pages, np.arange(len(pages))], 1).astype(np.int64)
            pools = [self.scratch[0], self.scratch[1]]
            pa.pa_read_pages_fp4(*pools, *self.pools, to_dev(pairs), device_errors=self.errs)
        pa.pa_prefill(out, q, *pools, to_dev(d_tables), to_dev(lens), to_dev(starts), D ** -0.5, HKV, MOST,
                      window=window, sinks=sinks, device_errors=self.errs)
        qh = rope_cases.values(storage_to_host(q, "bf16")).astype(np.float64)
        want, parts = oracle.prefill_f64(qh, *self.held(), tables, lens, starts, D ** -0.5, window, sinks)
        self.check(out, want, parts, 2.0 ** -8)

    def decode(self, ids, q, window, sinks):
        tables, lens = self.bm.build_block_tables(ids, MOST // BS)
        out = torch.full_like(q, float("nan"))
        call = pa.pa_decode_fp4 if self.fp4 else pa.pa_decode_window
        call(out, q, *self.pools, to_dev(tables), to_dev(lens), D ** -0.5, HKV, MOST, window=window, sinks=sinks,
             device_errors=self.errs)
        qh = rope_cases.values(storage_to_host(q, "bf16")).astype(np.float64)[:, None]
        want, parts = oracle.decode_window_f64(qh, *self.held(), tables, lens, D ** -0.5, window, sinks)
        self.check(out, want[:, 0], {k: v[:, 0] for k, v in parts.items()}, 2.0 ** -11 if self.fp4 else 2.0 ** -16)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_prompts_in_chunks_then_decode(fp4, window, sinks):
    loop = Loop(fp4)
    prompts = {1: [70, 64, 3], 2: [1, 40, 128], 3: [33, 0, 100]}
    had = dict.fromkeys(prompts, 0)
    for s in prompts:
        loop.bm.add_seq(s)
    for step in range(3):
        slots, pos, new = [], [], []
        for s, chunks in prompts.items():
            for _ in range(chunks[step]):
                slots.append(loop.bm.append_slot(s)[0])
                pos.append(had[s])
                had[s] += 1
            new.append(chunks[step])
        q = loop.append(slots, pos)
        loop.prompts(list(prompts), new, q, window, sinks)
    ids = list(prompts)
    for step in range(20):
        if step == 7:
            loop.bm.fork(1, 9)
            ids.append(9)
            had[9] = had[1]
        slots, pairs = loop.bm.append_slots(ids)
        if len(pairs):                                       # copy-on-write: rows with their scales are pages like any others
            pa.pa_copy_blocks(*loop.pools, to_dev(pairs), device_errors=loop.errs)
            oracle.copy_blocks(*loop.host, pairs)
        q = loop.append(slots, [had[s] for s in ids])
        for s in ids:
            had[s] += 1
        loop.decode(ids, q, window, sinks)
    for got, want in zip(loop.pools, loop.host):
        got = storage_to_host(got, "fp8" if fp4 else "bf16")
        if fp4:
            np.testing.assert_array_equal(oracle.unpack_rows(got), oracle.unpack_rows(want))
        else:
            np.testing.assert_array_equal(got, want)
    assert pa.pa_read_device_errors(loop.errs) == 0


def test_a_prompt_at_once_or_in_chunks():
    """Whole, or in pieces of any size: the same keys for each token, so the same result up to
    the order of the sums."""
    r = np.random.default_rng(31)
    T, nb = 700, 50
    k, v = (torch.from_numpy(r.standard_normal((nb, HKV, BS, D))).bfloat16().to(DEV) for _ in range(2))
    q = torch.from_numpy(r.standard_normal((T, HQ, D))).bfloat16().to(DEV)
    table = torch.from_numpy(r.permutation(nb).astype(np.int32))[None].to(DEV).contiguous()
    whole, parts = torch.empty_like(q), torch.empty_like(q)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    pa.pa_prefill(whole, q, k, v, table, i32(T), i32(0, T), D ** -0.5, HKV, T)
    at = 0
    for n in (1, 63, 64, 200, 7, 128, 237):
        pa.pa_prefill(parts[at:at + n], q[at:at + n], k, v, table, i32(at + n), i32(0, n), D ** -0.5, HKV, at + n)
        at += n
    assert at == T
    # each within half a step of the result and of the weights
    assert bool(((whole.double() - parts.double()).abs() <= 2 * (2.0 ** -8) * (whole.double().abs() + 1.0)).all())
    # the last token alone is a decode step
    out = torch.empty(1, HQ, D, dtype=torch.bfloat16, device=DEV)
    pa.pa_decode_window(out, q[-1:], k, v, table, i32(T), D ** -0.5, HKV, T, 0)
    assert bool(((out[0].double() - whole[-1].double()).abs() <= 2 * (2.0 ** -8) * (out[0].double().abs() + 1.0)).all())
