"""The decode step of a served model over a paged cache, operator by operator:

* ``rope``    -- rotary positions applied to q and k on the way into the cache
                 (pools in float32, bfloat16, or e4m3 with a fixed scale per kv head);
* ``window``  -- decode attention with a sliding window and a few first tokens that stay visible;
* ``append8`` -- the rotating append into e4m3 pools with a scale for each page and head;
* ``decode8`` -- decode attention over those pools (with or without a window).

Layouts are the library's: pools [blocks, kv heads, block size, head_dim], block tables by logical page.
Lengths belong to a case (``len_seed``); values, page order and slots follow ``prepare``'s seed.
"""
import math
import random

import torch

own = False

ROPE_BASE = 10000.0


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one user, one new token: nothing but latency
        dict(name="rope-one-token", op="rope", pool="bf16", tokens=1, seqs=1, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, bs=16, positions=32768, pads=0, len_seed=1),
        # a decode step of a batch padded to a captured size
        dict(name="rope-decode-batch", op="rope", pool="bf16", tokens=256, seqs=256, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, bs=16, positions=131072, pads=5, len_seed=2),
        # prompts being filled in, several at once
        dict(name="rope-prefill", op="rope", pool="bf16", tokens=16384, seqs=5, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, bs=16, positions=32768, pads=0, len_seed=3),
        # float32, heads rotated in part, neighbours paired, an odd number of tokens
        dict(name="rope-f32-partial", op="rope", pool="f32", tokens=777, seqs=9, hq=8, hkv=8, d=64, rot=32,
             interleaved=True, bs=16, positions=8192, pads=0, len_seed=4),
        # a small float32 model: short and long contexts around a short window
        dict(name="window-tiny-f32", op="window", pool="f32", seqs=4, q_len=1, hq=8, hkv=8, d=64, bs=16,
             lens="uniform", lo=17, hi=200, window=64, sinks=4, len_seed=5),
        # a windowed layer of a large ragged batch
        dict(name="window-gqa-batch", op="window", pool="bf16", seqs=256, q_len=1, hq=32, hkv=8, d=128, bs=16,
             lens="lognormal", lo=1024, hi=8192, window=1024, sinks=4, len_seed=6),
        # two drafted tokens verified far into long contexts whose middle pages are given back
        dict(name="window-verify-long", op="window", pool="bf16", seqs=16, q_len=2, hq=32, hkv=8, d=128, bs=32,
             lens="uniform", lo=100001, hi=131072, window=4096, sinks=4, len_seed=7),
        # a decode step's append: each sequence's last page holds earlier tokens
        dict(name="append8-decode-batch", op="append8", tokens=256, seqs=256, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, bs=16, positions=32768, pads=3, len_seed=8),
        # prompts filled in at once, pages ending inside and between them
        dict(name="append8-prefill", op="append8", tokens=8190, seqs=7, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, bs=16, positions=32768, pads=0, len_seed=9),
        # a few users' chat turns
        dict(name="decode8-small", op="decode8", seqs=4, q_len=1, hq=32, hkv=8, d=128, bs=16,
             lens="uniform", lo=17, hi=500, window=0, sinks=0, len_seed=10),
        # a large ragged batch
        dict(name="decode8-gqa-batch", op="decode8", seqs=256, q_len=1, hq=32, hkv=8, d=128, bs=16,
             lens="lognormal", lo=1024, hi=8192, window=0, sinks=0, len_seed=11),
        # a few very long contexts
        dict(name="decode8-long", op="decode8", seqs=4, q_len=1, hq=32, hkv=8, d=128, bs=32,
             lens="uniform", lo=131072, hi=131072, window=0, sinks=0, len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "window", "append8", "decode8"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32])
    if op in ("rope", "append8"):
        pool = rng.choice(["f32", "bf16", "bf16", "fp8"]) if op == "rope" else None
        d = rng.choice([64, 128]) if pool in ("f32", "bf16") else 128
        tokens = _log_int(rng, 1, 12000 if op == "rope" else 6000)
        pads = rng.choice([0, 0, min(tokens - 1, rng.randint(1, 7))])
        c = dict(op=op, tokens=tokens, seqs=_log_int(rng, 1, min(tokens - pads, 300)), hq=hkv * group, hkv=hkv, d=d,
                 rot=rng.choice([d, d, 16 * rng.randint(1, d // 16)]), interleaved=rng.random() < 0.4, bs=bs,
                 positions=32768, pads=pads, len_seed=rng.randrange(1 << 30))
        if pool:
            c["pool"] = pool
        return c
    q_len = rng.choice([1, 1, 1] + [n for n in (2, 4, 8) if n * group <= 8])
    seqs = _log_int(rng, 1, 300)
    most = max(8, min(100000, (1 << 21) // (seqs * hkv)))
    kind = rng.choice(["uniform", "lognormal"])
    hi = _log_int(rng, 8, most)
    lo = rng.randint(1, hi) if kind == "uniform" else max(1, hi // 8)
    windowed = op == "window" or rng.random() < 0.3
    c = dict(op=op, seqs=seqs, q_len=q_len, hq=hkv * group, hkv=hkv, d=128, bs=bs, lens=kind, lo=lo, hi=hi,
             window=_log_int(rng, 1, 6000) if windowed else 0,
             sinks=rng.choice([0, 1, 4, rng.randint(1, 80)]) if windowed else 0, len_seed=rng.randrange(1 << 30))
    if op == "window":
        c["pool"] = rng.choice(["f32", "bf16", "bf16"])
        c["d"] = rng.choice([64, 128])
    return c


def _lens(case):
    """Context lengths of a decode case: they count the q_len new tokens."""
    r = random.Random(case["len_seed"])
    lo, hi, q = case["lo"], case["hi"], case["q_len"]
    if case["lens"] == "uniform":
        return [max(q, r.randint(lo, hi)) for _ in range(case["seqs"])]
    return [max(q, min(hi, int(r.lognormvariate(math.log(lo), 1.0)) + 1)) for _ in range(case["seqs"])]


def _spans(case):
    """(earlier tokens, new tokens) of each sequence of an append: a decode step's sequences have a history
    of any length, a filled-in prompt starts anew or goes on where an earlier part of it ended."""
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


def _pow2_scale(amax):
    """The least power of two s with amax <= 448 s, from float32 amax (at least 2^-100)."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875).int()).clamp(min=-100))


def _e4m3(x):
    """Nearest e4m3 code (ties to even), magnitudes past 448 saturate."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _pool8(gen, nb, case):
    """An e4m3 pool with a power-of-two scale for each page and head; a few pages and columns are larger."""
    x = _randn(gen, nb, case["hkv"], case["bs"], case["d"])
    x *= torch.exp2(torch.randint(-2, 3, (nb, case["hkv"], 1, 1), generator=gen, device="cuda").float())
    x[..., :: 16] *= 4.0
    s = _pow2_scale(x.abs().amax((2, 3)))
    return _e4m3(x / s[..., None, None]), s


def _prepare_append(case, seed):
    gen, spans = _gen(seed), _spans(case)
    bs, hkv, hq, d = case["bs"], case["hkv"], case["hq"], case["d"]
    pos, slot_page, firsts, pages = [], [], [], 0
    for had, new in spans:
        p0, p1 = had // bs, (had + new - 1) // bs
        pos += range(had, had + new)
        slot_page += [pages + p // bs - p0 for p in range(had, had + new)]
        firsts.append(pages)
        pages += p1 - p0 + 1
    nb = pages + pages // 4 + 2                      # some pages belong to others
    order = torch.randperm(nb, generator=gen, device="cuda")
    pos, page = _ints(pos, torch.int64), _ints(slot_page, torch.int64)
    slots = order[page] * bs + pos % bs
    if case["pads"]:
        pad = torch.full((case["pads"],), -1, dtype=torch.int64, device="cuda")
        pos, slots = torch.cat([pos, pad]), torch.cat([slots, pad])
    pool = case.get("pool")
    dt = torch.float32 if pool == "f32" else torch.bfloat16
    qkv = _randn(gen, case["tokens"], (hq + 2 * hkv) * d).to(dt)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    st = dict(case=case, q=q, k=k, v=v, slots=slots, positions=pos, cos_sin=_table(case),
              q_out=torch.zeros(case["tokens"], hq, d, dtype=dt, device="cuda"),
              errors=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "append8":
        st["k_cache"], st["k_scales"] = _pool8(gen, nb, case)
        st["v_cache"], st["v_scales"] = _pool8(gen, nb, case)
    elif pool == "fp8":
        for n in ("k", "v"):
            st[n + "_scale"] = torch.rand(hkv, generator=gen, device="cuda") * 0.02 + 0.01
            st[n + "_cache"] = _e4m3(_randn(gen, nb, hkv, bs, d) / 0.02)
    else:
        for n in ("k", "v"):
            st[n + "_cache"] = _randn(gen, nb, hkv, bs, d).to(dt)
    return st


def _held(case, length):
    """Logical pages that a sequence still holds: those with a token that some new token sees."""
    bs = case["bs"]
    last = (length + bs - 1) // bs
    if not case["window"]:
        return list(range(last))
    lo = max(0, length - case["q_len"] + 1 - case["window"])
    return [p for p in range(last) if p * bs < case["sinks"] or (p + 1) * bs > lo]


def _prepare_decode(case, seed):
    gen, lens = _gen(seed), _lens(case)
    bs, hkv, hq, d = case["bs"], case["hkv"], case["hq"], case["d"]
    width = (max(lens) + bs - 1) // bs
    rows, cols = [], []
    for b, n in enumerate(lens):
        held = _held(case, n)
        rows += [b] * len(held)
        cols += held
    nb = len(rows) + len(rows) // 10 + 1
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(nb, generator=gen, device="cuda")
    tables[_ints(rows, torch.int64), _ints(cols, torch.int64)] = order[: len(rows)].int()
    dt = torch.float32 if case.get("pool") == "f32" else torch.bfloat16
    shape = (len(lens), case["q_len"], hq, d) if case["q_len"] > 1 else (len(lens), hq, d)
    st = dict(case=case, q=_randn(gen, *shape).to(dt), tables=tables, lens=_ints(lens, torch.int32), longest=max(lens),
              scale=d ** -0.5, errors=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "decode8":
        st["k_cache"], st["k_scales"] = _pool8(gen, nb, case)
        st["v_cache"], st["v_scales"] = _pool8(gen, nb, case)
    else:
        for n in ("k", "v"):
            st[n + "_cache"] = torch.empty(nb, hkv, bs, d, dtype=dt, device="cuda").normal_(generator=gen)
    return st


def prepare(case, seed):
    return _prepare_append(case, seed) if case["op"] in ("rope", "append8") else _prepare_decode(case, seed)


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


def _plain_append(st):
    case, bs = st["case"], st["case"]["bs"]
    live = (st["positions"] >= 0).nonzero()[:, 0]
    slots = st["slots"][live]
    rows = st["cos_sin"][st["positions"][live]]
    st["q_out"][live] = _rotate(st["q"][live].float(), rows, case).to(st["q_out"].dtype)
    k, v = _rotate(st["k"][live].float(), rows, case), st["v"][live].float()
    page, off = slots // bs, slots % bs
    if case["op"] == "append8":
        _plain_write8(st["k_cache"], st["k_scales"], k, page, off)
        _plain_write8(st["v_cache"], st["v_scales"], v, page, off)
    elif case["pool"] == "fp8":
        st["k_cache"].view(torch.uint8)[page, :, off] = _e4m3(k / st["k_scale"][None, :, None]).view(torch.uint8)
        st["v_cache"].view(torch.uint8)[page, :, off] = _e4m3(v / st["v_scale"][None, :, None]).view(torch.uint8)
    else:
        st["k_cache"][page, :, off] = k.to(st["k_cache"].dtype)
        st["v_cache"][page, :, off] = v.to(st["v_cache"].dtype)


def _plain_write8(cache, scales, x, page, off):
    """Rows x [T, H, D] into slots (page, off): the page's scale grows to hold them, and what it holds follows."""
    codes = cache.view(torch.uint8)
    amax = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(2), "amax")
    fresh = torch.zeros(scales.shape[0], dtype=torch.bool, device=scales.device)
    fresh[page[off == 0]] = True
    need = _pow2_scale(amax)
    new = torch.where(fresh[:, None], need, torch.maximum(scales, need))[page]
    ratio = (scales[page] / new)[:, :, None, None]
    kept = codes[page].view(torch.float8_e4m3fn).float() * ratio
    codes[page] = torch.where(fresh[page][:, None, None, None], codes[page], _e4m3(kept).view(torch.uint8))
    codes[page, :, off] = _e4m3(x / new[:, :, None]).view(torch.uint8)
    scales[page] = new


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
    bs, hkv, d, q_len = case["bs"], case["hkv"], case["d"], case["q_len"]
    pos = _visible(st)
    there = pos < lens[:, None]
    pos = torch.where(there, pos, 0)
    page = st["tables"].long().gather(1, pos // bs).clamp(min=0)
    if case["op"] == "decode8":
        k, v = (st[n + "_cache"].view(torch.uint8)[page, :, pos % bs].view(torch.float8_e4m3fn).float()
                * st[n + "_scales"][page][..., None] for n in ("k", "v"))
    else:
        k, v = (st[n + "_cache"][page, :, pos % bs].float() for n in ("k", "v"))
    # rows: the group's heads of each kv head, for each new token
    q = st["q"].float().view(len(lens), q_len, hkv, -1, d).permute(0, 2, 1, 3, 4)
    s = torch.matmul(q.flatten(2, 3), k.permute(0, 2, 3, 1)).unflatten(2, (q_len, -1)) * st["scale"]
    at = lens[:, None] - q_len + torch.arange(q_len, device="cuda")
    seen = there[:, None] & (pos[:, None] <= at[..., None])
    if case["window"]:
        seen &= (at[..., None] - pos[:, None] < case["window"]) | (pos[:, None] < case["sinks"])
    s = s.masked_fill(~seen[:, None, :, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).unflatten(2, (q_len, -1))
    return o.permute(0, 2, 1, 3, 4).reshape(st["q"].shape).to(st["q"].dtype)


# --------------------------------------------------------------------------- the framework's calls
def _own_append(st):
    import paged_kv_cache_190_gb300 as pa
    case = st["case"]
    args = (st["q_out"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"], st["positions"], st["cos_sin"])
    if case["op"] == "append8":
        pa.pa_rope_and_cache_fp8_block(*args, st["k_scales"], st["v_scales"], interleaved=case["interleaved"],
                                       device_errors=st["errors"])
    elif case["pool"] == "fp8":
        pa.pa_rope_and_cache_fp8(*args, st["k_scale"], st["v_scale"], interleaved=case["interleaved"],
                                 device_errors=st["errors"])
    else:
        pa.pa_rope_and_cache(*args, interleaved=case["interleaved"], device_errors=st["errors"])


def _own_decode(st):
    import paged_kv_cache_190_gb300 as pa
    case = st["case"]
    out = torch.empty_like(st["q"])
    if "workspace" not in st:                       # scratch that a serving loop keeps
        size = pa.pa_decode_window_workspace_size(case["seqs"], case["q_len"] * case["hq"], case["hkv"], case["d"],
                                                  case["bs"], st["longest"], case["window"], case["sinks"])
        st["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    if case["op"] == "decode8":
        return pa.pa_decode_fp8_block(out, st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"],
                                      st["k_scales"], st["v_scales"], case["hkv"], st["longest"], window=case["window"],
                                      sinks=case["sinks"], workspace=st["workspace"], device_errors=st["errors"])
    return pa.pa_decode_window(out, st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"],
                               case["hkv"], st["longest"], case["window"], case["sinks"], workspace=st["workspace"],
                               device_errors=st["errors"])


def run(state):
    if state["case"]["op"] in ("window", "decode8"):
        return _own_decode(state) if own else _plain_decode(state)
    if own:
        _own_append(state)
    else:
        _plain_append(state)
    return {n: state[n] for n in ("q_out", "k_cache", "v_cache", "k_scales", "v_scales") if n in state}


# --------------------------------------------------------------------------- cost and definition
def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] in ("rope", "append8"):
        pool = case.get("pool", "fp8")
        e, e_pool = (4, 4) if pool == "f32" else (2, 2) if pool == "bf16" else (2, 1)
        n = case["tokens"] - case["pads"]
        spans = _spans(case)
        seen = set()
        for had, new in spans:
            seen.update(range(had, had + new))
        total = n * (2 * hq * d * e + 2 * hkv * d * (e + e_pool)) + 16 * case["tokens"] + 4 * case["rot"] * len(seen)
        if case["op"] == "append8":
            bs = case["bs"]
            pages = sum((had + new - 1) // bs - had // bs + 1 for had, new in spans)
            kept = sum(had % bs > 0 for had, _ in spans)
            total += 8 * hkv * (pages + kept)       # scales written, and read where a page goes on
        return {"bytes": total, "flops": 3 * case["rot"] * n * (hq + hkv)}
    e, e_pool = (4, 4) if case.get("pool") == "f32" else (2, 2) if case["op"] == "window" else (2, 1)
    tokens = pairs = pages = 0
    for n in _lens(case):
        if case["window"]:
            far = n - case["q_len"] + 1 - case["window"]
            see = n - max(0, far - case["sinks"]) if far > 0 else n
        else:
            see = n
        tokens += see
        pages += len(_held(case, n))
        for j in range(case["q_len"]):
            m = n - case["q_len"] + j + 1
            pairs += min(m, case["window"] + min(case["sinks"], max(0, m - case["window"]))) if case["window"] else m
    total = tokens * 2 * hkv * d * e_pool + 2 * case["seqs"] * case["q_len"] * hq * d * e + 4 * pages + 4 * case["seqs"]
    if case["op"] == "decode8":
        total += 8 * hkv * pages
    return {"bytes": total, "flops": 4 * d * hq * pairs}


def _nearest_e4m3(x):
    """Values of the nearest e4m3 numbers of float64 x: three fraction bits, steps of 2^-9 at the least."""
    step = torch.exp2((torch.frexp(x.abs())[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(case, seed):
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
    q = torch.cat([turned(st["q"][:n], turn), torch.zeros_like(st["q_out"][n:], dtype=torch.float64)])
    out = {"q_out": q}
    slots = st["slots"][:n]
    for name, x in (("k", turned(st["k"][:n], turn)), ("v", st["v"][:n].double())):
        cache = st[name + "_cache"]
        rows = cache.float().double().transpose(1, 2).flatten(0, 1)      # [slots, heads, d]
        if case["op"] == "append8":
            scales = st[name + "_scales"].double()
            page = slots // bs
            need = torch.zeros_like(scales)
            need.scatter_reduce_(0, page[:, None].expand(-1, case["hkv"]), x.abs().amax(-1), "amax")
            least = torch.exp2(torch.ceil(torch.log2((need / 448.0).clamp(min=2.0 ** -100))))
            touched, begun = torch.zeros(len(scales), dtype=torch.bool, device="cuda"), torch.zeros(len(scales), dtype=torch.bool, device="cuda")
            touched[page] = True
            begun[slots[slots % bs == 0] // bs] = True
            grown = torch.where(begun[:, None], least, torch.maximum(least, scales))
            grown = torch.where(touched[:, None], grown, scales)
            kept = _nearest_e4m3(rows.unflatten(0, (-1, bs)) * (scales / grown)[:, None, :, None])
            move = (touched & ~begun)[:, None, None, None]
            rows = torch.where(move, kept, rows.unflatten(0, (-1, bs))).flatten(0, 1)
            rows[slots] = _nearest_e4m3(x / grown[page][..., None])
            out[name + "_scales"] = grown
        elif case["pool"] == "fp8":
            rows[slots] = _nearest_e4m3(x / st[name + "_scale"].double()[:, None])
        else:
            rows[slots] = x
        out[name + "_cache"] = rows.unflatten(0, (-1, bs)).transpose(1, 2)
    return out


def _exact_decode(case, seed):
    st = prepare(case, seed)
    bs, hkv, d, q_len = case["bs"], case["hkv"], case["d"], case["q_len"]
    group = case["hq"] // hkv
    out = torch.zeros(case["seqs"], q_len, hkv, group, d, dtype=torch.float64, device="cuda")
    q = st["q"].double().view(out.shape)
    for b, n in enumerate(_lens(case)):
        at = torch.tensor([t for p in _held(case, n) for t in range(p * bs, min(n, (p + 1) * bs))], device="cuda")
        page = st["tables"][b].long()[at // bs]
        kv = []
        for name in ("k", "v"):
            x = st[name + "_cache"].view(torch.uint8)[page, :, at % bs].view(torch.float8_e4m3fn).double() if case["op"] == "decode8" \
                else st[name + "_cache"][page, :, at % bs].double()
            kv.append(x * st[name + "_scales"].double()[page][..., None] if case["op"] == "decode8" else x)
        for j in range(q_len):
            here = n - q_len + j
            sel = at <= here
            if case["window"]:
                sel &= (at > here - case["window"]) | (at < case["sinks"])
            w = torch.softmax(torch.einsum("hgd,thd->hgt", q[b, j], kv[0][sel]) * st["scale"], -1)
            out[b, j] = torch.einsum("hgt,thd->hgd", w, kv[1][sel])
    return out.view(st["q"].shape)


def exact(case, seed):
    return _exact_append(case, seed) if case["op"] in ("rope", "append8") else _exact_decode(case, seed)
