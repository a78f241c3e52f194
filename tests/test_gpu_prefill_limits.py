"""The prompt attention where calls are refused, cut short or very long: starts that make
sequences claim each other's rows, data errors in any sequence, waits that expire and waits
that rightly take long."""
import numpy as np
import pytest
import torch

import paged_kv_cache_190_gb300 as pa
from gpu_helpers import DEV
from prefill_cases import Prompts
from test_gpu_prefill import Dev, check

pytestmark = pytest.mark.gpu


def _swinging(tokens, seqs):
    """0, T, 0, T, ...: each other sequence claims every row, the ones between decrease."""
    return torch.arange(seqs + 1, dtype=torch.int32, device=DEV) % 2 * tokens


# (type, query heads of the one kv head, head_dim, rows of a tile, tokens, sequences)
CLAIMS = [("bf16", 8, 64, 256, 600, 400), ("f32", 8, 64, 64, 900, 700), ("bf16", 1, 128, 256, 90, 3000),
          ("bf16", 8, 64, 256, 371000, 371001), ("f32", 8, 64, 64, 186000, 186001)]


@pytest.mark.parametrize("dtype,hq,d,rows,tokens,seqs", CLAIMS)
def test_starts_that_claim_more_tiles_than_there_are_rows(dtype, hq, d, rows, tokens, seqs):
    """Reported, however many tiles the sequences claim together (the last two cases: more than
    31 bits), and rows are left as they were or are one of their sequences' (zeros, as the
    pools are)."""
    claimed = (seqs + 1) // 2 * -(-tokens * hq // rows)
    assert tokens < 100000 or claimed > 2 ** 31 - 1
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = torch.zeros(tokens, hq, d, dtype=tdt, device=DEV)
    out = torch.full_like(q, 7.0)
    pools = [torch.zeros(2, 1, 16, d, dtype=tdt, device=DEV) for _ in range(2)]
    tables = torch.zeros(seqs, 1, dtype=torch.int32, device=DEV)
    lens = torch.full((seqs,), 16, dtype=torch.int32, device=DEV)
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_prefill(out, q, *pools, tables, lens, _swinging(tokens, seqs), d ** -0.5, 1, 16, device_errors=errs)
    assert pa.pa_read_device_errors(errs) == pa.PA_DEVERR_BAD_LENGTH
    assert bool(((out == 7.0) | (out == 0.0)).all())


def test_swinging_starts_leave_the_workspace_usable():
    c = Prompts(70, "bf16", [40, 3, 300, 20], [0, 900, 10, 0], 8, 2, 128, 16)
    ws = torch.empty(pa.pa_prefill_workspace_size(c.rows, 400, 8, 2, 128), dtype=torch.uint8, device=DEV)
    dv = Dev(c)
    pa.pa_prefill(dv.out, dv.q, dv.kc, dv.vc, dv.tables[:1].repeat(400, 1), dv.lens[:1].repeat(400), _swinging(c.rows, 400),
                  c.scale, c.hkv, int(c.lens.max()), workspace=ws, device_errors=dv.errs)
    assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH
    dv.out.fill_(7.0)
    dv.call(workspace=ws)
    assert dv.errors() == 0
    check(c, dv.out)


# ------------------------------------------------- data errors without a plan
def _single(seed, dtype, seqs, empty=0):
    """Sequences of one new token each (and `empty` without any) behind a few earlier ones."""
    r = np.random.default_rng(seed)
    new = np.concatenate([np.ones(seqs, int), np.zeros(empty, int)])
    return Prompts(seed, dtype, new, r.integers(0, 30, len(new)), 1, 1, 64, 16, before=1, behind=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs,empty", [(40, 0), (100, 0), (3, 90), (33, 31)])
def test_data_errors_in_any_sequence_are_reported(dtype, seqs, empty):
    """Calls small enough to go without a plan: the last sequence's errors are seen as the
    first one's are, and the other sequences keep their results."""
    c = _single(71 + seqs, dtype, seqs, empty)
    ref = Dev(c)
    ref.call()
    assert ref.errors() == 0
    check(c, ref.out)
    n, most = len(c.lens), int(c.lens.max())
    for b in (0, 31, 32, n // 2, n - 1):
        if b >= n:
            continue
        r0, r1 = int(c.starts[b]), int(c.starts[b + 1])
        others = torch.ones(c.rows, dtype=torch.bool, device=DEV)
        others[r0:r1] = False
        for bad in (-1, most + 1) + ((0,) if r1 > r0 else ()):
            dv = Dev(c)
            dv.lens[b] = bad
            dv.call(max_context_len=most)
            # (a length that is clamped reaches table entries that are no pages)
            assert dv.errors() & pa.PA_DEVERR_BAD_LENGTH, f"length {bad} of sequence {b}"
            assert torch.equal(dv.out[others], ref.out[others])
    for start in (c.rows + 1, int(c.starts[-2]) - 1):
        dv = Dev(c)
        dv.starts[-1] = start
        dv.call()
        assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH, f"last start {start}"


# ------------------------------------------------------------------ long waits
@pytest.fixture
def wait_limit():
    yield pa.pa_debug_set_wait_limit
    pa.pa_debug_set_wait_limit(-1)


def _pools(hkv, d, pages, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.empty(pages, hkv, 16, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(2)]


def _limited(wait_limit, polls, out, *args, **kw):
    errs = torch.zeros(1, dtype=torch.int32, device=DEV)
    wait_limit(polls)
    pa.pa_prefill(out, *args, device_errors=errs, **kw)
    flags = pa.pa_read_device_errors(errs)
    wait_limit(-1)
    return flags


@pytest.mark.parametrize("d", [64, 128])
def test_a_short_prompt_behind_a_long_document(d, wait_limit):
    """The document's length is aligned, so no V row of it has to be cleared until the short
    prompt's turn comes, milliseconds later.  64 polls are about 0.24 ms: more than any single
    step takes, less than the document."""
    T, short, h = 65536, 20, 8
    k, v = _pools(h, d, T // 16 + 2, 74)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table = torch.full((2, T // 16), -1, dtype=torch.int32, device=DEV)
    table[0] = torch.arange(T // 16, device=DEV)
    table[1, :2] = i32(T // 16, T // 16 + 1)
    q = torch.randn(T + short, h, d, device=DEV).bfloat16()
    args = (q, k, v, table, i32(T, short), i32(0, T, T + short), d ** -0.5, h, T)
    want, got = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    assert _limited(wait_limit, -1, want, *args) == 0
    assert _limited(wait_limit, 64, got, *args) == 0
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
def test_halves_without_rows_for_long(d, wait_limit):
    """Chunks of at most 128 rows leave the second half of an item's rows without work until
    the whole tiles of a fresh prompt come, which are shorter and so last."""
    n, chunk, had, fresh, h = 160, 100, 8092, 2048, 8
    pages = (had + chunk + 15) // 16
    k, v = _pools(h, d, pages + fresh // 16, 75)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(n + 1, 1)      # (all chunks behind one context)
    table[n, :fresh // 16] = pages + torch.arange(fresh // 16, dtype=torch.int32, device=DEV)
    q = torch.randn(n * chunk + fresh, h, d, device=DEV).bfloat16()
    args = (q, k, v, table, i32([had + chunk] * n + [fresh]), i32([chunk * i for i in range(n + 1)] + [len(q)]),
            d ** -0.5, h, had + chunk)
    want, got = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    assert _limited(wait_limit, -1, want, *args) == 0
    assert _limited(wait_limit, 64, got, *args) == 0
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))


# ---------------------------------------------------------------- expired waits
@pytest.mark.parametrize("d,bs,new,had,window,sinks", [
    (128, 16, [600, 33], [0, 900], 0, 0), (128, 32, [20], [0], 0, 0), (128, 16, [130], [20000], 0, 0),
    (64, 16, [100], [6000], 0, 0), (64, 32, [300, 77, 5], [0, 500, 3000], 100, 20)])
def test_no_polls_at_all(d, bs, new, had, window, sinks, wait_limit):
    """With a limit of 0 the kernel gives up with its first copies in flight: reported, and the
    next call as ever."""
    c = Prompts(72, "bf16", new, had, 8, 2, d, bs, window, sinks)
    dv = Dev(c)
    ws = torch.zeros(pa.pa_prefill_workspace_size(c.rows, len(new), 8, 2, d), dtype=torch.uint8, device=DEV)
    for _ in range(5):
        wait_limit(0)
        for _ in range(3):
            dv.call(workspace=ws)
        assert dv.errors() == pa.PA_DEVERR_TIMEOUT
        wait_limit(-1)
        dv.out.fill_(7.0)
        dv.call(workspace=ws)
        assert dv.errors() == 0
        check(c, dv.out)


@pytest.mark.parametrize("d", [64, 128])
def test_a_call_that_waits_for_nothing_expires_nowhere(d, wait_limit):
    """Rows that see nothing need no copy and no product: they are zeros under any limit."""
    c = Prompts(73, "bf16", [40, 300], [0, 0], 8, 2, d, 16)
    dv = Dev(c)
    dv.lens.zero_()
    wait_limit(0)
    dv.call()
    assert dv.errors() == pa.PA_DEVERR_BAD_LENGTH and bool((dv.out == 0).all())
