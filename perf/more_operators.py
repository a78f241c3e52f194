"""Prompts over a paged cache, and a cache in four bits, operator by operator:

* ``prefill`` -- causal attention of whole prompts, or of the next chunks of prompts, over the paged cache that
                 their keys and values stand in: sequences of different lengths packed one after another
                 (pools in float32 or bfloat16; with or without a sliding window and first tokens);
* ``store4``  -- the rotating append into pools of 4-bit codes with a scale for each 16 columns, and the touched
                 pages read back in bfloat16 for a prompt's attention;
* ``read4``   -- whole contexts read back from such pools;
* ``decode4`` -- decode attention over such pools (with or without a window).

Layouts are the library's: pools [blocks, kv heads, block size, head_dim], block tables by logical page. A row of
a 4-bit pool is 72 bytes: 64 of e2m1 codes (column 2 i in the low half of byte i), then 8 scales, one for 16
columns: the upper bits of a positive half (5 of exponent, 3 of fraction; byte b is the half with the bits b << 7).
Lengths belong to a case (``len_seed``); values, page order and slots follow ``prepare``'s seed.
"""
import math
import random

import torch

own = False

ROPE_BASE = 10000.0
LEAST_STEP = -17                                    # log2 of the smallest scale
MOST_SCALE = 10240.0                                # the largest scale: 6 of it is a half


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one short question
        dict(name="prefill-one-short", op="prefill", pool="bf16", seqs=1, hq=32, hkv=8, d=128, bs=16,
             new="uniform", q_lo=37, q_hi=37, had_lo=0, had_hi=0, window=0, sinks=0, pads=0, len_seed=21),
        # a small float32 model: a few prompts, some of them going on
        dict(name="prefill-tiny-f32", op="prefill", pool="f32", seqs=5, hq=8, hkv=8, d=64, bs=16,
             new="uniform", q_lo=17, q_hi=200, had_lo=0, had_hi=100, window=0, sinks=0, pads=3, len_seed=22),
        # prompts of a busy server, packed: a few long ones among many shorter
        dict(name="prefill-prompts", op="prefill", pool="bf16", seqs=12, hq=32, hkv=8, d=128, bs=16,
             new="lognormal", q_lo=700, q_hi=4096, had_lo=0, had_hi=0, window=0, sinks=0, pads=5, len_seed=23),
        # the next chunks of prompts that are filled in piece by piece
        dict(name="prefill-chunks", op="prefill", pool="bf16", seqs=6, hq=32, hkv=8, d=128, bs=16,
             new="uniform", q_lo=200, q_hi=512, had_lo=1000, had_hi=15000, window=0, sinks=0, pads=0, len_seed=24),
        # a windowed layer with narrow heads, each head its own keys
        dict(name="prefill-window", op="prefill", pool="bf16", seqs=4, hq=16, hkv=16, d=64, bs=32,
             new="uniform", q_lo=1500, q_hi=5000, had_lo=0, had_hi=3000, window=1024, sinks=4, pads=0, len_seed=25),
        # one long document
        dict(name="prefill-long", op="prefill", pool="bf16", seqs=1, hq=32, hkv=8, d=128, bs=16,
             new="uniform", q_lo=16384, q_hi=16384, had_lo=0, had_hi=0, window=0, sinks=0, pads=0, len_seed=26),
        # a decode step's append
        dict(name="store4-decode-batch", op="store4", tokens=256, seqs=256, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, bs=16, positions=32768, pads=3, len_seed=27),
        # prompts filled in at once, pages ending inside and between them
        dict(name="store4-prefill", op="store4", tokens=8190, seqs=7, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, bs=16, positions=32768, pads=0, len_seed=28),
        # one user's earlier turns
        dict(name="read4-turns", op="read4", seqs=1, hq=32, hkv=8, d=128, bs=16, lens="uniform", lo=523, hi=523,
             len_seed=29),
        # the contexts of a batch of prompts that go on
        dict(name="read4-contexts", op="read4", seqs=8, hq=32, hkv=8, d=128, bs=32, lens="uniform", lo=1000, hi=16384,
             len_seed=30),
        # a few users' chat turns
        dict(name="decode4-small", op="decode4", seqs=4, q_len=1, hq=32, hkv=8, d=128, bs=16,
             lens="uniform", lo=17, hi=500, window=0, sinks=0, len_seed=31),
        # a large ragged batch
        dict(name="decode4-gqa-batch", op="decode4", seqs=256, q_len=1, hq=32, hkv=8, d=128, bs=16,
             lens="lognormal", lo=1024, hi=8192, window=0, sinks=0, len_seed=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "store4", "read4", "decode4"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32])
    c = dict(op=op, hq=hkv * group, hkv=hkv, d=128, bs=bs, len_seed=rng.randrange(1 << 30))
    if op == "prefill":
        c["pool"] = rng.choice(["f32", "bf16", "bf16", "bf16"])
        c["d"] = rng.choice([64, 128])
        c["seqs"] = _log_int(rng, 1, 48)
        pairs = (1 << 27 if c["pool"] == "f32" else 1 << 31) // (c["seqs"] * c["hq"])
        q_hi = _log_int(rng, 1, max(2, min(8000, math.isqrt(pairs))))
        c["new"] = rng.choice(["uniform", "lognormal"])
        c["q_lo"] = rng.randint(0, q_hi) if c["new"] == "uniform" else max(1, q_hi // 6)
        c["q_hi"] = q_hi
        c["had_hi"] = rng.choice([0, _log_int(rng, 1, max(2, min(40000, pairs // q_hi - q_hi)))])
        c["had_lo"] = rng.randint(0, c["had_hi"])
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 5000)])
        c["sinks"] = rng.choice([0, 1, 4, rng.randint(1, 200)]) if c["window"] else 0
        c["pads"] = rng.choice([0, 0, rng.randint(1, 9)])
        return c
    if op == "store4":
        c["tokens"] = _log_int(rng, 1, 6000)
        c["pads"] = rng.choice([0, 0, min(c["tokens"] - 1, rng.randint(1, 7))])
        c["seqs"] = _log_int(rng, 1, min(c["tokens"] - c["pads"], 300))
        c["rot"] = rng.choice([128, 128, 16 * rng.randint(1, 8)])
        c["interleaved"] = rng.random() < 0.4
        c["positions"] = 32768
        return c
    c["seqs"] = _log_int(rng, 1, 300 if op == "decode4" else 40)
    most = max(8, min(100000, ((1 << 21) if op == "decode4" else (1 << 20)) // (c["seqs"] * hkv)))
    c["lens"] = rng.choice(["uniform", "lognormal"])
    c["hi"] = _log_int(rng, 8, most)
    c["lo"] = rng.randint(1, c["hi"]) if c["lens"] == "uniform" else max(1, c["hi"] // 8)
    if op == "decode4":
        c["q_len"] = rng.choice([1, 1, 1] + [n for n in (2, 4, 8) if n * group <= 8])
        windowed = rng.random() < 0.3
        c["window"] = _log_int(rng, 1, 6000) if windowed else 0
        c["sinks"] = rng.choice([0, 1, 4, rng.randint(1, 80)]) if windowed else 0
    return c


def _spread(r, kind, lo, hi):
    return r.randint(lo, hi) if kind == "uniform" else min(hi, int(r.lognormvariate(math.log(lo), 1.0)) + 1)


def _lens(case):
    """Context lengths of a decode or a read; a decode's count the q_len new tokens."""
    r = random.Random(case["len_seed"])
    return [max(case.get("q_len", 1), _spread(r, case["lens"], case["lo"], case["hi"])) for _ in range(case["seqs"])]


def _prompts(case):
    """(earlier tokens, new tokens) of each sequence of a prefill."""
    r = random.Random(case["len_seed"])
    return [(r.randint(case["had_lo"], case["had_hi"]), _spread(r, case["new"], case["q_lo"], case["q_hi"]))
            for _ in range(case["seqs"])]


def _spans(case):
    """(earlier tokens, new tokens) of each sequence of an append: a decode step's sequences have a history of any
    length, a filled-in prompt starts anew or goes on where an earlier part of it ended."""
    r = random.Random(case["len_seed"])
    n, s = case["tokens"] - case["pads"], case["seqs"]
    cuts = sorted(r.sample(range(1, n), s - 1)) if s < n else list(range(1, n))
    new = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    room = case["positions"] - n
    return [(0 if m > 1 and r.random() < 0.5 else r.randint(0, room), m) for m in new]


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _ints(v, dtype):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _table(case):
    """cos | sin of position times frequency, one float32 row for each position."""
    half = case["rot"] // 2
    freq = ROPE_BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(case["positions"], dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _scale_of(amax):
    """The nearest scale to amax / 6 (ties to even): three bits of fraction, steps of 2^-17 at the least."""
    y = amax / 6.0
    step = torch.exp2((torch.frexp(y)[1] - 4).clamp(min=LEAST_STEP).to(y.dtype))
    return (torch.round(y / step) * step).clamp(max=MOST_SCALE)


def _nearest_e2m1(z):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to |z| with z's sign, ties to the even code."""
    a = z.abs().clamp(max=6.0)
    step = torch.exp2((torch.frexp(a)[1] - 1).clamp(0, 2).to(z.dtype) - 1)
    return torch.copysign(torch.round(a / step) * step, z)


def _pack4(x):
    """Rows [..., 128] in float32 as rows of 72 bytes."""
    b = x.unflatten(-1, (8, 16))
    s = _scale_of(b.abs().amax(-1))
    v = _nearest_e2m1(torch.where(s[..., None] > 0, b / s[..., None], 0.0)).flatten(-2)
    a = v.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(v).to(torch.uint8)
    low, high = code.unflatten(-1, (64, 2)).unbind(-1)
    return torch.cat([low + high * 16, (s.half().view(torch.int16) >> 7).to(torch.uint8)], -1)


def _unpack4(rows, dtype=torch.float32):
    """Rows of 72 bytes as the values [..., 128] that they stand for."""
    code = torch.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).flatten(-2)
    m = (code & 7).to(dtype)
    v = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(code > 7, -v, v)
    s = (rows[..., 64:].to(torch.int16) << 7).view(torch.float16).to(dtype)
    return (v.unflatten(-1, (8, 16)) * s[..., None]).flatten(-2)


def _pool4(gen, nb, case):
    """A 4-bit pool: rows of different sizes, a few columns larger than the others."""
    pool = torch.empty(nb, case["hkv"], case["bs"], 72, dtype=torch.uint8, device="cuda")
    for part in pool.split(max(1, (1 << 20) // (case["hkv"] * case["bs"]))):
        x = _randn(gen, *part.shape[:3], 128)
        x *= torch.exp2(torch.randint(-2, 3, (*part.shape[:3], 1), generator=gen, device="cuda").float())
        x[..., ::16] *= 4.0
        part.copy_(_pack4(x))
    return pool


def _prepare_append(case, seed):
    gen, spans = _gen(seed), _spans(case)
    bs, hkv, hq, d = case["bs"], case["hkv"], case["hq"], case["d"]
    pos, slot_page, pages = [], [], 0
    for had, new in spans:
        p0, p1 = had // bs, (had + new - 1) // bs
        pos += range(had, had + new)
        slot_page += [pages + p // bs - p0 for p in range(had, had + new)]
        pages += p1 - p0 + 1
    nb = pages + pages // 4 + 2                     # some pages belong to others
    order = torch.randperm(nb, generator=gen, device="cuda")
    pos, page = _ints(pos, torch.int64), _ints(slot_page, torch.int64)
    slots = order[page] * bs + pos % bs
    if case["pads"]:
        pad = torch.full((case["pads"],), -1, dtype=torch.int64, device="cuda")
        pos, slots = torch.cat([pos, pad]), torch.cat([slots, pad])
    qkv = _randn(gen, case["tokens"], (hq + 2 * hkv) * d).bfloat16()
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    pairs = torch.stack([order[:pages], torch.arange(pages, device="cuda")], 1)
    back = torch.zeros(2, pages, hkv, bs, d, dtype=torch.bfloat16, device="cuda")
    return dict(case=case, q=q, k=k, v=v, slots=slots, positions=pos, cos_sin=_table(case), pairs=pairs,
                q_out=torch.zeros(case["tokens"], hq, d, dtype=torch.bfloat16, device="cuda"),
                k_cache=_pool4(gen, nb, case), v_cache=_pool4(gen, nb, case), k_back=back[0], v_back=back[1],
                errors=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_read(case, seed):
    gen = _gen(seed)
    pages = sum((n + case["bs"] - 1) // case["bs"] for n in _lens(case))
    nb = pages + pages // 4 + 2
    order = torch.randperm(nb, generator=gen, device="cuda")
    back = torch.zeros(2, pages, case["hkv"], case["bs"], case["d"], dtype=torch.bfloat16, device="cuda")
    return dict(case=case, pairs=torch.stack([order[:pages], torch.arange(pages, device="cuda")], 1),
                k_cache=_pool4(gen, nb, case), v_cache=_pool4(gen, nb, case), k_back=back[0], v_back=back[1],
                errors=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _held(case, length, new):
    """Logical pages that a sequence still holds: those with a token that some new token sees."""
    bs = case["bs"]
    last = (length + bs - 1) // bs
    if not case["window"]:
        return list(range(last))
    lo = max(0, length - new + 1 - case["window"])
    return [p for p in range(last) if p * bs < case["sinks"] or (p + 1) * bs > lo]


def _paged(case, gen, lens, new):
    """(block tables, blocks of the pool): the held pages in a random order, the other entries -1."""
    rows, cols = [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        held = _held(case, n, m)
        rows += [b] * len(held)
        cols += held
    nb = len(rows) + len(rows) // 10 + 1
    tables = torch.full((len(lens), max(1, (max(lens) + case["bs"] - 1) // case["bs"])), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(nb, generator=gen, device="cuda")
    tables[_ints(rows, torch.int64), _ints(cols, torch.int64)] = order[: len(rows)].int()
    return tables, nb


def _prepare_prefill(case, seed):
    gen, prompts = _gen(seed), _prompts(case)
    lens, new = [a + n for a, n in prompts], [n for _, n in prompts]
    hkv, hq, d, bs = case["hkv"], case["hq"], case["d"], case["bs"]
    tables, nb = _paged(case, gen, lens, new)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    dt = torch.float32 if case["pool"] == "f32" else torch.bfloat16
    rows = starts[-1] + case["pads"]
    st = dict(case=case, q=_randn(gen, rows, hq, d).to(dt), tables=tables, lens=_ints(lens, torch.int32),
              starts=_ints(starts, torch.int32), longest=max(lens), most_new=max(new), scale=d ** -0.5,
              out=torch.zeros(rows, hq, d, dtype=dt, device="cuda"),
              errors=torch.zeros(1, dtype=torch.int32, device="cuda"))
    for n in ("k", "v"):
        st[n + "_cache"] = torch.empty(nb, hkv, bs, d, dtype=dt, device="cuda").normal_(generator=gen)
    return st


def _prepare_decode(case, seed):
    gen, lens = _gen(seed), _lens(case)
    hq, d = case["hq"], case["d"]
    tables, nb = _paged(case, gen, lens, [case["q_len"]] * len(lens))
    shape = (len(lens), case["q_len"], hq, d) if case["q_len"] > 1 else (len(lens), hq, d)
    return dict(case=case, q=_randn(gen, *shape).bfloat16(), tables=tables, lens=_ints(lens, torch.int32),
                longest=max(lens), scale=d ** -0.5, k_cache=_pool4(gen, nb, case), v_cache=_pool4(gen, nb, case),
                errors=torch.zeros(1, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    return {"prefill": _prepare_prefill, "store4": _prepare_append, "read4": _prepare_read,
            "decode4": _prepare_decode}[case["op"]](case, seed)


# --------------------------------------------------------------------------- plain forms
def _rotate(x, rows, case):
    """x [T, H, D] in float32 with the first `rot` columns of each head rotated; rows: the tokens' table rows."""
    rot, half = case["rot"], case["rot"] // 2
    cos, sin = rows[:, None, :half], rows[:, None, half:]
    y = x.clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
    a, b = x[..., one], x[..., two]
    y[..., one] = a * cos - b * sin
    y[..., two] = b * cos + a * sin
    return y


def _plain_read(st):
    src, dst = st["pairs"].unbind(1)
    st["k_back"][dst] = _unpack4(st["k_cache"][src]).to(torch.bfloat16)
    st["v_back"][dst] = _unpack4(st["v_cache"][src]).to(torch.bfloat16)


def _plain_store(st):
    case, bs = st["case"], st["case"]["bs"]
    live = (st["positions"] >= 0).nonzero()[:, 0]
    slots = st["slots"][live]
    rows = st["cos_sin"][st["positions"][live]]
    st["q_out"][live] = _rotate(st["q"][live].float(), rows, case).to(torch.bfloat16)
    st["k_cache"][slots // bs, :, slots % bs] = _pack4(_rotate(st["k"][live].float(), rows, case))
    st["v_cache"][slots // bs, :, slots % bs] = _pack4(st["v"][live].float())
    _plain_read(st)


def _weights(s, seen):
    """Softmax of s [..., rows, t] over the seen t, in place; rows that see nothing are zeros."""
    s.masked_fill_(~seen, -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    return s.div_(s.sum(-1, keepdim=True).clamp(min=1e-30))


def _plain_prefill(st):
    case, lens = st["case"], st["lens"].long()
    bs, hkv, hq, d = case["bs"], case["hkv"], case["hq"], case["d"]
    first, n = st["starts"][:-1].long(), st["starts"].long().diff()
    j = torch.arange(max(1, st["most_new"]), device="cuda")
    there = j < n[:, None]                          # [B, Q]
    row = torch.where(there, first[:, None] + j, 0)
    t = torch.arange(st["longest"], device="cuda")
    page = st["tables"].long()[:, t // bs].clamp(min=0)
    k, v = (st[c + "_cache"][page, :, t % bs].float() for c in ("k", "v"))       # [B, T, Hkv, D]
    q = st["q"][row].float().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)      # [B, Hkv, Q, G, D]
    s = torch.matmul(q.flatten(2, 3), k.permute(0, 2, 3, 1)).mul_(st["scale"]).unflatten(2, (len(j), -1))
    at = (lens - n)[:, None] + j
    seen = t <= at[..., None]
    if case["window"]:
        seen &= (at[..., None] - t < case["window"]) | (t < case["sinks"])
    p = _weights(s, (seen & there[..., None])[:, None, :, None])
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).unflatten(2, (len(j), -1))
    out = st["out"]
    out[row[there]] = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[there].to(out.dtype)
    return out


def _visible(st):
    """Positions that the new tokens of each sequence may see, [B, N] (those past the end are masked later)."""
    case, lens = st["case"], st["lens"].long()
    if not case["window"]:
        return torch.arange(st["longest"], device="cuda").expand(len(lens), -1)
    span = min(case["window"] + case["q_len"] - 1, st["longest"])
    lo = (lens - span).clamp(min=0)
    sinks = torch.arange(min(case["sinks"], st["longest"]), device="cuda").expand(len(lens), -1)
    tail = lo[:, None] + torch.arange(span, device="cuda")
    return torch.cat([torch.where(sinks < lo[:, None], sinks, st["longest"]), tail], 1)


def _plain_decode(st):
    case, lens = st["case"], st["lens"].long()
    bs, hkv, q_len = case["bs"], case["hkv"], case["q_len"]
    pos = _visible(st)
    there = pos < lens[:, None]
    pos = torch.where(there, pos, 0)
    page = st["tables"].long().gather(1, pos // bs).clamp(min=0)
    k, v = (_unpack4(st[c + "_cache"][page, :, pos % bs]) for c in ("k", "v"))
    # rows: the group's heads of each kv head, for each new token
    q = st["q"].float().view(len(lens), q_len, hkv, -1, case["d"]).permute(0, 2, 1, 3, 4)
    s = torch.matmul(q.flatten(2, 3), k.permute(0, 2, 3, 1)).mul_(st["scale"]).unflatten(2, (q_len, -1))
    at = lens[:, None] - q_len + torch.arange(q_len, device="cuda")
    seen = there[:, None] & (pos[:, None] <= at[..., None])
    if case["window"]:
        seen &= (at[..., None] - pos[:, None] < case["window"]) | (pos[:, None] < case["sinks"])
    p = _weights(s, seen[:, None, :, None])
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).unflatten(2, (q_len, -1))
    return o.permute(0, 2, 1, 3, 4).reshape(st["q"].shape).to(torch.bfloat16)


# --------------------------------------------------------------------------- the framework's calls
def _own_prefill(st):
    import paged_kv_cache_190_gb300 as pa
    case = st["case"]
    if "workspace" not in st:                       # scratch that a serving loop keeps
        size = pa.pa_prefill_workspace_size(len(st["q"]), case["seqs"], case["hq"], case["hkv"], case["d"])
        st["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return pa.pa_prefill(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["starts"],
                         st["scale"], case["hkv"], st["longest"], window=case["window"], sinks=case["sinks"],
                         workspace=st["workspace"], device_errors=st["errors"])


def _own_read(st):
    import paged_kv_cache_190_gb300 as pa
    pa.pa_read_pages_fp4(st["k_back"], st["v_back"], st["k_cache"], st["v_cache"], st["pairs"],
                         device_errors=st["errors"])


def _own_store(st):
    import paged_kv_cache_190_gb300 as pa
    pa.pa_rope_and_cache_fp4(st["q_out"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"],
                             st["positions"], st["cos_sin"], interleaved=st["case"]["interleaved"],
                             device_errors=st["errors"])
    _own_read(st)


def _own_decode(st):
    import paged_kv_cache_190_gb300 as pa
    case = st["case"]
    out = torch.empty_like(st["q"])
    if "workspace" not in st:
        size = pa.pa_decode_window_workspace_size(case["seqs"], case["q_len"] * case["hq"], case["hkv"], case["d"],
                                                  case["bs"], st["longest"], case["window"], case["sinks"])
        st["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return pa.pa_decode_fp4(out, st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"],
                            case["hkv"], st["longest"], window=case["window"], sinks=case["sinks"],
                            workspace=st["workspace"], device_errors=st["errors"])


def run(state):
    op = state["case"]["op"]
    if op == "prefill":
        return _own_prefill(state) if own else _plain_prefill(state)
    if op == "decode4":
        return _own_decode(state) if own else _plain_decode(state)
    if op == "store4":
        if own:
            _own_store(state)
        else:
            _plain_store(state)
    elif own:
        _own_read(state)
    else:
        _plain_read(state)
    return {n: state[n] for n in ("q_out", "k_back", "v_back") if n in state}


# --------------------------------------------------------------------------- cost and definition
def _seen(case, length, new):
    """(tokens that some new token sees, pairs of a new token and a token that it sees)."""
    w, s = case["window"], case["sinks"]
    if not w:
        return (length if new else 0), new * (length - new) + new * (new + 1) // 2
    pairs = 0
    for m in range(length - new + 1, length + 1):
        pairs += m if m <= w else w + min(s, m - w)
    far = length - new + 1 - w
    return ((length - max(0, far - s) if far > 0 else length) if new else 0), pairs


def work(case):
    d, hq, hkv, bs = case["d"], case["hq"], case["hkv"], case["bs"]
    if case["op"] == "prefill":
        e = 4 if case["pool"] == "f32" else 2
        tokens = pairs = pages = rows = 0
        for had, new in _prompts(case):
            t, p = _seen(case, had + new, new)
            tokens, pairs, rows = tokens + t, pairs + p, rows + new
            pages += len(_held(case, had + new, new)) if new else 0
        return {"bytes": tokens * 2 * hkv * d * e + 2 * rows * hq * d * e + 4 * (pages + 2 * case["seqs"] + 1),
                "flops": 4 * d * hq * pairs}
    if case["op"] == "store4":
        n, spans = case["tokens"] - case["pads"], _spans(case)
        angles = set()
        for had, new in spans:
            angles.update(range(had, had + new))
        pages = sum((had + new - 1) // bs - had // bs + 1 for had, new in spans)
        total = n * (4 * hq * d + 4 * hkv * d + 2 * 72 * hkv) + 16 * case["tokens"] + 4 * case["rot"] * len(angles)
        total += 16 * pages + 2 * pages * hkv * bs * 2 * d + 2 * 72 * hkv * (pages * bs - n)   # the other rows are read
        return {"bytes": total, "flops": 3 * case["rot"] * n * (hq + hkv) + 4 * n * hkv * d + 2 * pages * hkv * bs * d}
    if case["op"] == "read4":
        rows = sum((n + bs - 1) // bs for n in _lens(case)) * bs * hkv
        return {"bytes": 2 * rows * (72 + 2 * d) + 16 * (rows // (bs * hkv)), "flops": 2 * rows * d}
    tokens = pairs = pages = 0
    for n in _lens(case):
        t, p = _seen(case, n, case["q_len"])
        tokens, pairs = tokens + t, pairs + p
        pages += len(_held(case, n, case["q_len"]))
    total = tokens * 2 * hkv * 72 + 2 * case["seqs"] * case["q_len"] * hq * d * 2 + 4 * pages + 4 * case["seqs"]
    return {"bytes": total, "flops": 4 * d * hq * pairs}


def _values4(rows):
    """What 72-byte rows stand for, by looking the codes up."""
    look = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=rows.device)
    look = torch.cat([look, -look])
    b = rows[..., :64].long()
    v = look[torch.stack([b % 16, b // 16], -1)].flatten(-2)
    u = rows[..., 64:].double()
    e, f = torch.floor(u / 8), u % 8
    s = torch.where(e > 0, (8 + f) * torch.exp2(e - 18), f * 2.0 ** -17)
    return v * s.repeat_interleave(16, -1)


def _quantised4(x):
    """float64 rows [..., 128] as the values that they are stored as."""
    b = x.unflatten(-1, (8, 16))
    y = (b.abs().amax(-1) / 6.0).clamp(min=2.0 ** -60)
    step = torch.exp2(torch.floor(torch.log2(y)).clamp(min=-14.0) - 3)
    s = (torch.round(y / step) * step).clamp(max=MOST_SCALE)[..., None]
    z = torch.where(s > 0, b / torch.where(s > 0, s, 1.0), 0.0)
    a = z.abs()
    low = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a.clamp(max=6.0) / 2)))
    return (torch.sign(z) * low * s).flatten(-2)


def _exact_store(case, seed):
    st = prepare(case, seed)
    bs, rot, half = case["bs"], case["rot"], case["rot"] // 2

    def turned(x, turn):
        x = x.double()
        pairs = x[..., :rot].unflatten(-1, (half, 2)) if case["interleaved"] else x[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., rot:]], -1)

    n = case["tokens"] - case["pads"]               # padding comes last
    row = st["cos_sin"].double()[st["positions"][:n]]
    turn = torch.complex(row[:, :half], row[:, half:])[:, None]
    out = {"q_out": torch.cat([turned(st["q"][:n], turn), torch.zeros_like(st["q_out"][n:], dtype=torch.float64)])}
    slots = st["slots"][:n]
    for name, x in (("k", turned(st["k"][:n], turn)), ("v", st["v"][:n].double())):
        rows = _values4(st[name + "_cache"]).transpose(1, 2).flatten(0, 1)       # [slots, heads, d]
        rows[slots] = _quantised4(x)
        back = rows.unflatten(0, (-1, bs)).transpose(1, 2)
        out[name + "_back"] = torch.zeros_like(st[name + "_back"], dtype=torch.float64)
        out[name + "_back"][st["pairs"][:, 1]] = back[st["pairs"][:, 0]]
    return out


def _exact_read(case, seed):
    st = prepare(case, seed)
    out = {}
    for name in ("k", "v"):
        out[name + "_back"] = torch.zeros_like(st[name + "_back"], dtype=torch.float64)
        out[name + "_back"][st["pairs"][:, 1]] = _values4(st[name + "_cache"][st["pairs"][:, 0]])
    return out


def _attend(case, q, table, had, rows_of, scale):
    """q [n, Hkv, G, D] in 64 bits: the new tokens behind `had` earlier ones. rows_of(page, offset) gives (K, V)."""
    bs, n = case["bs"], q.shape[0]
    at = torch.tensor([t for p in _held(case, had + n, n) for t in range(p * bs, min(had + n, (p + 1) * bs))], device="cuda")
    k, v = rows_of(table.long()[at // bs], at % bs)
    out = torch.empty_like(q)
    for i in range(0, n, 1024):
        here = had + torch.arange(i, min(n, i + 1024), device="cuda")
        sel = at <= here[:, None]
        if case["window"]:
            sel &= (at > here[:, None] - case["window"]) | (at < case["sinks"])
        hi = int((at <= int(here[-1])).sum())       # none of these rows sees what is behind
        for h in range(case["hkv"]):
            s = torch.einsum("ngd,td->ngt", q[i:i + 1024, h], k[:hi, h]) * scale
            w = torch.softmax(s.masked_fill(~sel[:, None, :hi], -math.inf), -1)
            out[i:i + 1024, h] = torch.einsum("ngt,td->ngd", w, v[:hi, h])
    return out


def _exact_prefill(case, seed):
    st = prepare(case, seed)
    out = st["out"].double()
    at = 0
    for b, (had, new) in enumerate(_prompts(case)):
        if new:
            q = st["q"][at:at + new].double().unflatten(1, (case["hkv"], -1))
            o = _attend(case, q, st["tables"][b], had, lambda p, i: (st["k_cache"][p, :, i].double(), st["v_cache"][p, :, i].double()), st["scale"])
            out[at:at + new] = o.flatten(1, 2)
        at += new
    return out


def _exact_decode(case, seed):
    st = prepare(case, seed)
    q = st["q"].double().view(case["seqs"], case["q_len"], case["hkv"], -1, case["d"])
    out = torch.empty_like(q)
    for b, n in enumerate(_lens(case)):
        out[b] = _attend(case, q[b], st["tables"][b], n - case["q_len"],
                         lambda p, i: (_values4(st["k_cache"][p, :, i]), _values4(st["v_cache"][p, :, i])), st["scale"])
    return out.view(st["q"].shape)


def exact(case, seed):
    if case["op"] == "prefill" and 8 * case["d"] * case["hq"] * sum(_seen(case, a + n, n)[1] for a, n in _prompts(case)) > 12e12:
        return None
    return {"prefill": _exact_prefill, "store4": _exact_store, "read4": _exact_read, "decode4": _exact_decode}[case["op"]](case, seed)
