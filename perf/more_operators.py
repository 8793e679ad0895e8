"""A key-value cache in 4 bits, measured: its block tables, its write and reading back, the attention over it.

The cache lies in pages of `page` tokens.  Every row (page, head, place) of keys and of values is `dim` values as
FP4 E2M1 pairs (uint8, the first value in the low nibble) with one E8M0 scale byte (2^(byte - 127), 255 a NaN) for
every 32 of them: scale 2^(floor(log2 max|x|) - 2), values rounded to nearest even, saturating at 6.  A request's
tokens lie in the pages that its row of the block table names; a slot is page * page_size + place.

With `own` false `run` computes the plain forms from elementary torch operations; with `own` true it calls the
library.  Heads and lengths are those of the package's workloads (32 heads of queries, 8 of keys, 128 values,
32768 tokens) and odd neighbours.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 32
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # a decoding step's bookkeeping: 64 requests, one new token each, some requests done
        {"name": "tables_step", "op": "tables", "batch": 64, "longest": 8192, "new": 1, "page": 64, "spare": 1.0},
        # 512 prompts of up to 512 tokens taken in at once, in small pages, more of them than pages are left
        {"name": "tables_prompts", "op": "tables", "batch": 512, "longest": 4096, "new": 512, "page": 16, "spare": 0.97},
        # the new keys and values of a decoding step
        {"name": "cache_step", "op": "cache", "tokens": 64, "kv_heads": 8, "dim": 128, "page": 64, "type": "bf16"},
        # FP32 rows of three blocks, an odd number of heads, tokens without a place among them
        {"name": "cache_ragged", "op": "cache", "tokens": 1531, "kv_heads": 5, "dim": 96, "page": 16, "type": "fp32"},
        # a prompt batch's keys and values
        {"name": "cache_prompt", "op": "cache", "tokens": 32768, "kv_heads": 8, "dim": 128, "page": 64, "type": "bf16"},
        # one request's next token: latency
        {"name": "attend_token", "op": "attend", "batch": 1, "longest": 1000, "new": 1, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "type": "bf16", "lse": False},
        # a serving batch's next tokens, requests of all lengths up to 8192 and an empty one
        {"name": "attend_batch", "op": "attend", "batch": 64, "longest": 8192, "new": 1, "ragged": True, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "type": "bf16", "lse": False},
        # two requests at the cache's full length, to be joined with another part's result by the sums' logarithms
        {"name": "attend_long", "op": "attend", "batch": 2, "longest": 32768, "new": 1, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "type": "bf16", "lse": True},
        # drafted tokens of 32 requests looked at together, small heads, a window
        {"name": "attend_drafts", "op": "attend", "batch": 32, "longest": 4099, "new": 5, "ragged": True, "heads": 24,
         "kv_heads": 3, "dim": 64, "page": 32, "window": 1024, "type": "bf16", "lse": False},
        # FP32 queries, heads of three blocks, odd lengths
        {"name": "attend_ragged", "op": "attend", "batch": 7, "longest": 1021, "new": 77, "ragged": True, "heads": 10,
         "kv_heads": 5, "dim": 96, "page": 16, "window": 0, "type": "fp32", "lse": True},
        # the next 2048 tokens of a long prompt
        {"name": "attend_chunk", "op": "attend", "batch": 1, "longest": 18432, "new": 2048, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "type": "bf16", "lse": False},
        # a whole prompt
        {"name": "attend_prompt", "op": "attend", "batch": 1, "longest": 8192, "new": 8192, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "type": "bf16", "lse": False},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["tables", "cache", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        batch = _spread(rng, 1, 1024)
        return {"op": op, "batch": batch, "longest": _spread(rng, 64, 16384), "new": _spread(rng, 1, max(1, 131072 // batch)),
                "page": page, "spare": rng.choice([0.5, 0.9, 1.0, 1.0])}
    heads, dim = rng.choice([1, 2, 3, 5, 8, 8, 16]), 32 * rng.choice([1, 2, 3, 4, 4, 6, 8])
    if op == "cache":
        return {"op": op, "tokens": min(_spread(rng, 1, 32768), 32768 * 1024 // (heads * dim)), "kv_heads": heads, "dim": dim,
                "page": page, "type": rng.choice(["bf16", "fp32"])}
    group = rng.choice([1, 2, 4, 4, 6, 8])
    longest = _spread(rng, 1, 32768)
    # keys and values of the longest listed batch, and the pairs and products of the longest listed prompt, are not passed
    batch = min(_spread(rng, 1, 128), max(1, 64 * 8192 * 1024 // (longest * heads * dim)))
    new = rng.choice([1, 1, rng.randint(2, 8), _spread(rng, 1, 8192)])
    new = max(1, min(new, longest, 8192 * 8192 * 32 // (batch * longest * heads * group) * 128 // max(128, dim)))
    return {"op": op, "batch": batch, "longest": longest, "new": new, "ragged": rng.random() < 0.7, "heads": heads * group,
            "kv_heads": heads, "dim": dim, "page": page, "window": rng.choice([0, 0, 0, _spread(rng, 1, 8192)]),
            "type": rng.choice(["bf16", "bf16", "fp32"]), "lse": rng.random() < 0.5}


def _lengths(case):
    """Lengths (with the new tokens) and new tokens of the requests, by the case alone."""
    rng = random.Random("%d %d %d" % (case["batch"], case["longest"], case["new"]))
    batch, longest, new = case["batch"], case["longest"], case["new"]
    if case["op"] == "tables":
        return [rng.randint(0, longest) for _ in range(batch)], [new if new == 1 else rng.randint(0, new) for _ in range(batch)]
    if not case["ragged"]:
        return [longest] * batch, [min(new, longest)] * batch
    lens = [longest] + [rng.randint(0, longest) for _ in range(batch - 1)]
    if batch > 3:
        lens[2] = 0
    if new == 1:
        return lens, [1] * batch
    return lens, [min(n, rng.randint(1, new)) for n in lens]


def _done(case):
    """Requests that end before a step, by the case alone."""
    rng = random.Random("done %d %d" % (case["batch"], case["longest"]))
    return [rng.random() < 0.06 for _ in range(case["batch"])]


def work(case):
    if case["op"] == "tables":
        lens, add = _lengths(case)
        done = _done(case)
        add = [0 if d else a for a, d in zip(add, done)]
        p = case["page"]
        need = sum(-(-(n + a) // p) - -(-n // p) for n, a in zip(lens, add))
        freed = sum(-(-n // p) for n, d in zip(lens, done) if d)
        # lengths, new tokens and flags in, lengths and starts out; pages moved; slot and position of each token
        return {"bytes": 21 * len(lens) + 8 * (need + freed) + 8 * sum(add), "flops": 0}
    if case["op"] == "cache":
        n = case["tokens"] * case["kv_heads"] * case["dim"] * 2
        item = 2 if case["type"] == "bf16" else 4
        # in, codes and scales, and the values that they stand for out
        return {"bytes": n * item + n // 2 + n // BLOCK + n * 2, "flops": 6 * n}
    lens, add = _lengths(case)
    item = 2 if case["type"] == "bf16" else 4
    window = case["window"] or case["longest"]
    pairs = keys = 0
    for length, new in zip(lens, add):
        first = max(0, length - new)
        keys += length - max(0, first - window + 1) if length else 0
        # rows at positions first .. length - 1 see min(position + 1, window) keys
        full = max(0, min(length, window) - first)
        pairs += full * (2 * first + full + 1) // 2 + (length - first - full) * window
    rows = sum(add) * case["heads"]
    return {"bytes": keys * case["kv_heads"] * (case["dim"] + case["dim"] // 16) + 2 * rows * case["dim"] * item
            + (4 * rows if case["lse"] else 0), "flops": 4 * case["dim"] * case["heads"] * pairs}


# -------------------------------------------------------------- plain forms --
def _scale_of(byte):
    """2^(byte - 127) in FP32 from the bits: byte 0 is the subnormal 2^-127, 255 a NaN."""
    b = byte.to(torch.int32)
    bits = torch.where(b == 0, torch.full_like(b, 0x00400000), b << 23)
    return torch.where(b == 255, torch.full_like(b, 0x7FC00000), bits).view(torch.float32)


def _quantize(x):
    """FP32 rows [..., dim] -> E2M1 pairs [..., dim / 2] and scale bytes [..., dim / 32]."""
    v = x.unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1)
    fine = torch.isfinite(top)
    exponent = torch.frexp(torch.where(fine, top, torch.ones_like(top)))[1] - 1
    byte = torch.where(top == 0, 0, (exponent + 125).clamp(0, 254))
    v = v * ((254 - byte).to(torch.int32) << 23).view(torch.float32).unsqueeze(-1)
    a = v.abs()
    # steps of 1/2 under 2, of 1 under 4, of 2 above, to the even multiple
    code = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a * 0.5) + 4).clamp(max=7))
    code = torch.where(fine.unsqueeze(-1), code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3), 0)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.where(fine, byte, 255).to(torch.uint8)


def _values(codes, scales):
    """Codes [..., dim / 2] and scale bytes [..., dim / 32] as FP32 rows."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = grid[torch.stack([codes & 15, codes >> 4], -1).to(torch.int32).flatten(-2)]
    return (v.unflatten(-1, (-1, BLOCK)) * _scale_of(scales.view(torch.uint8)).unsqueeze(-1)).flatten(-2)


def _tables(state):
    """Pages of requests that are done go back; then every request gets the pages that its new tokens need."""
    p, table, free, left = state["page"], state["table"], state["free"], state["n_free"].long()
    width = table.shape[1]
    column = torch.arange(width, device=table.device)
    # back onto the stack of free pages, request after request
    lens = state["lens"].long()
    back = torch.where(state["done"], (lens + p - 1) // p, 0)
    at = left + (back.cumsum(0) - back).unsqueeze(1) + column
    at = torch.where(column < back.unsqueeze(1), at, free.numel())
    free = torch.cat([free, free.new_zeros(1)]).scatter(0, at.flatten(), table.flatten())[:-1]
    left = left + back.sum()
    lens = torch.where(state["done"], 0, lens)
    # from the top of the stack
    add = state["add"].long()
    starts = torch.cat([add.new_zeros(1), add.cumsum(0)])
    have, want = (lens + p - 1) // p, (lens + add + p - 1) // p
    fits = (want <= width) & (starts[1:] <= state["tokens"])
    need = torch.where(fits, want - have, 0)
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= left))
    taken = torch.where(served & (need > 0), upto, 0).amax()
    first = (upto - need).unsqueeze(1) + column - have.unsqueeze(1)
    new = served.unsqueeze(1) & (column >= have.unsqueeze(1)) & (column < want.unsqueeze(1))
    table = torch.where(new, free[(left - 1 - first).clamp(0, free.numel() - 1)], table)
    # each token's request, position and slot
    t = torch.arange(state["tokens"], device=table.device)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True).clamp(max=add.numel() - 1)
    live = (t < starts[-1]) & served[b]
    position = torch.where(live, lens[b] + t - starts[b], 0)
    slot = torch.where(live, table[b, position // p].long() * p + position % p, -1)
    i32 = torch.int32
    return [torch.where(served, lens + add, lens).to(i32), starts.to(i32), slot.to(i32), position.to(i32),
            (left - taken).to(i32), table, free]


def _cache(state):
    got = []
    slots = state["slots"].long()
    live = slots >= 0
    page, place = slots.clamp(min=0) // state["page"], slots.clamp(min=0) % state["page"]
    for name in ("k", "v"):
        codes, scales = _quantize(state[name].float())
        # rows without a slot write back what is there, at the place of the first row that has one
        codes = torch.where(live.view(-1, 1, 1), codes, codes[state["first"]])
        scales = torch.where(live.view(-1, 1, 1), scales, scales[state["first"]])
        at = (torch.where(live, page, page[state["first"]]), slice(None), torch.where(live, place, place[state["first"]]))
        state["cache"][name][at] = codes
        state["cache"][name + "_scales"][at] = scales
        back = _values(state["cache"][name][at], state["cache"][name + "_scales"][at])
        got.append(torch.where(live.view(-1, 1, 1), back, 0).to(torch.bfloat16))
    return got


def _attend(state):
    q, c, lens = state["q"], state["cache"], state["lens"].long()
    batch, tall, group = lens.numel(), state["most"], q.shape[1] // c["k"].shape[1]
    starts = state["starts"]
    starts = torch.arange(batch + 1, device=q.device) if starts is None else starts.long()
    count = starts[1:] - starts[:-1]
    # keys and values of every request, its pages side by side: [batch, kv heads, keys, dim]
    pages = state["table"].long()
    k, v = (_values(c[n][pages], c[n + "_scales"][pages]).transpose(1, 2).flatten(2, 3) for n in ("k", "v"))
    # queries filled up to the most of a request: [batch, kv heads, group * tall, dim]
    i = torch.arange(tall, device=q.device)
    row = (starts[:-1].unsqueeze(1) + i).clamp(max=max(0, q.shape[0] - 1))
    x = q[row].float().unflatten(2, (-1, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = torch.matmul(x, k.transpose(2, 3)) * (1.0 / math.sqrt(q.shape[2]))
    at = (lens - count).unsqueeze(1) + i
    key = torch.arange(k.shape[2], device=q.device)
    seen = (key <= at.unsqueeze(2)) & (key < lens.view(-1, 1, 1))
    if state["window"]:
        seen &= key > (at - state["window"]).unsqueeze(2)
    seen = seen.unsqueeze(1).unsqueeze(2)
    s = torch.where(seen, s.unflatten(2, (group, tall)), -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, 0, top))
    total = e.sum(-1, keepdim=True)
    # behind a request's end the pages hold what they held: no key of them counts
    v = torch.where((key < lens.view(-1, 1)).view(batch, 1, -1, 1), v, 0)
    y = torch.matmul(e.flatten(2, 3), v).unflatten(2, (group, tall)) / torch.where(total == 0, 1, total)
    lse = torch.log(total) + top
    # rows back to where the queries lie
    t = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True).clamp(max=batch - 1)
    out = y.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, t - starts[b]].to(q.dtype)
    if not state["lse"]:
        return out
    return [out, lse.squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[b, t - starts[b]]]


# ------------------------------------------------------------------ prepare --
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _keys(shape, g):
    """N(0, 1) with a few channels larger than the rest, as keys have them."""
    loud = 1 + 4 * (torch.rand(shape[-2:], device="cuda", generator=g) < 0.04).float()
    return torch.randn(shape, device="cuda", generator=g) * loud


def _some(shape, g):
    """N(0, 1) around a mean of each channel, as values have them."""
    return torch.randn(shape, device="cuda", generator=g) + 0.3 * torch.randn(shape[-2:], device="cuda", generator=g)


def _table(lens, page, n_pages, width, g):
    """Pages dealt to requests in a random order: (table with pages of other requests behind the lengths, pages left)."""
    order = torch.randperm(n_pages, device="cuda", generator=g)
    used = torch.tensor([-(-n // page) for n in lens], device="cuda")
    first = (used.cumsum(0) - used).unsqueeze(1) + torch.arange(width, device="cuda")
    return order[first % n_pages].to(torch.int32), order[int(used.sum()):].to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    state = dict(case)
    page = case["page"]
    if case["op"] == "tables":
        lens, add = _lengths(case)
        done = _done(case)
        add = [0 if d else a for a, d in zip(add, done)]
        used = sum(-(-n // page) for n in lens)
        need = sum(-(-(n + a) // page) - -(-n // page) for n, a in zip(lens, add))
        freed = sum(-(-n // page) for n, d in zip(lens, done) if d)
        n_pages = used + max(1, int(case["spare"] * need) - freed)
        state["table"], left = _table(lens, page, n_pages, max(1, -(-(case["longest"] + case["new"]) // page)), g)
        state["free"] = torch.cat([left, _ints([-1] * (n_pages - left.numel()))])
        state["n_free"], state["n_pages"] = _ints([left.numel()]), n_pages
        state["lens"], state["add"] = _ints(lens), _ints(add)
        state["done"] = torch.tensor(done, device="cuda")
        state["tokens"] = max(1, sum(add))
        return state
    heads, dim = case["kv_heads"], case["dim"]
    if case["op"] == "cache":
        tokens = case["tokens"]
        n_pages = -(-tokens // page) + 3
        state["k"] = _keys((tokens, heads, dim), g).to(TORCH[case["type"]])
        state["v"] = _some((tokens, heads, dim), g).to(TORCH[case["type"]])
        slots = torch.randperm(n_pages * page, device="cuda", generator=g)[:tokens].to(torch.int32)
        if tokens > 100:
            slots[3::50] = -1
        state["slots"], state["first"], state["n_pages"] = slots, 0, n_pages
        state["cache"] = _empty(n_pages, heads, page, dim)
        return state
    lens, add = _lengths(case)
    n_pages = sum(-(-n // page) for n in lens) + 2
    state["table"], _ = _table(lens, page, n_pages, max(1, -(-case["longest"] // page)), g)
    state["cache"] = cache = _empty(n_pages, heads, page, dim)
    step = max(1, (1 << 27) // (heads * page * dim))
    for at in range(0, n_pages, step):  # pages at a time, for the memory
        n = min(step, n_pages - at)
        cache["k"][at:at + n], cache["k_scales"][at:at + n] = _quantize(_keys((n, page, heads, dim), g).transpose(1, 2))
        cache["v"][at:at + n], cache["v_scales"][at:at + n] = _quantize(_some((n, page, heads, dim), g).transpose(1, 2))
    state["q"] = (1.5 * torch.randn(sum(add), case["heads"], dim, device="cuda", generator=g)).to(TORCH[case["type"]])
    state["lens"], state["most"] = _ints(lens), max(add)
    starts = [0]
    for a in add:
        starts.append(starts[-1] + a)
    state["starts"] = None if case["new"] == 1 else _ints(starts)
    return state


def _empty(n_pages, heads, page, dim):
    """A cache of zeros."""
    made = {}
    for name in ("k", "v"):
        made[name] = torch.zeros(n_pages, heads, page, dim // 2, dtype=torch.uint8, device="cuda")
        made[name + "_scales"] = torch.zeros(n_pages, heads, page, dim // BLOCK, dtype=torch.uint8, device="cuda")
    return made


# ---------------------------------------------------------------------- run --
def run(state):
    if own:
        return _run_own(state)
    return {"tables": _tables, "cache": _cache, "attend": _attend}[state["op"]](state)


def _run_own(state):
    from lossless_float_weight_amd import zn
    if state["op"] == "tables":
        lens, left = zn.kv_release(state["lens"], state["done"], state["table"], state["free"], state["n_free"], state["page"])
        step = zn.kv_extend(lens, state["add"], state["table"], state["free"], left, state["page"], state["n_pages"],
                            state["tokens"])
        return [step.lens, step.starts, step.slots, step.positions, step.n_free, state["table"], state["free"]]
    c = state["cache"]
    cache = zn.MxCache(c["k"], c["k_scales"], c["v"], c["v_scales"])
    if state["op"] == "cache":
        zn.mx_kv_write(state["k"], state["v"], cache, state["slots"])
        # what the 4 bits stand for, as a user reads it back
        return list(zn.mx_kv_read(cache, state["slots"], dtype=torch.bfloat16))
    got = zn.mx_attention(state["q"], cache, state["table"], state["lens"], starts=state["starts"],
                          max_new=state["most"], window=state["window"], lse=state["lse"])
    return list(got) if state["lse"] else got


# -------------------------------------------------------------------- exact --
GRID64 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def _quantize64(x):
    """The values that rows [..., dim] have in 4 bits, in 64 bits: the grid searched for the nearest."""
    v = x.double().unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1, keepdim=True)
    powers = torch.tensor([math.ldexp(1.0, e) for e in range(-127, 128)], dtype=torch.float64, device=x.device)
    at = torch.bucketize(top, powers, right=True) - 1
    scale = powers[(at - 2).clamp(min=0)]
    grid = torch.tensor(GRID64, dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    a = (v / scale).abs()
    i = torch.bucketize(a, middle)
    tie = (i < 7) & (a == middle[i.clamp(max=6)])
    i = i + (tie & (i % 2 == 1)).to(i.dtype)
    return (torch.copysign(grid[i], v) * scale).flatten(-2)


def _values64(codes, scales):
    grid = torch.tensor(GRID64 + [-x for x in GRID64], dtype=torch.float64, device=codes.device)
    c = codes.long()
    v = grid[torch.stack([c % 16, c // 16], -1).flatten(-2)]
    return (v.unflatten(-1, (-1, BLOCK)) * torch.pow(2.0, scales.double() - 127).unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers, which have to be equal
    state = prepare(case, seed)
    if case["op"] == "cache":
        live = (state["slots"] >= 0).view(-1, 1, 1)
        return [torch.where(live, _quantize64(state[n]), 0) for n in ("k", "v")]
    lens, add = _lengths(case)
    q, c, page = state["q"], state["cache"], case["page"]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    table, at = state["table"].tolist(), 0
    for row, length, new in zip(table, lens, add):
        pages = torch.tensor(row[:-(-length // page)], device="cuda", dtype=torch.long)
        for h in range(case["kv_heads"] if length else 0):
            k, v = (_values64(c[n][pages, h], c[n + "_scales"][pages, h]).flatten(0, 1)[:length] for n in ("k", "v"))
            for first in range(0, new, 1024):  # rows at a time, for the memory
                x = q[at + first:at + min(new, first + 1024), h * group:(h + 1) * group].double()
                s = torch.einsum("ngd,kd->ngk", x, k) / math.sqrt(case["dim"])
                own_place = torch.arange(length - new + first, length - new + first + x.shape[0], device="cuda").view(-1, 1, 1)
                key = torch.arange(length, device="cuda")
                hidden = key > own_place
                if case["window"]:
                    hidden = hidden | (key <= own_place - case["window"])
                s.masked_fill_(hidden, -math.inf)
                rows = slice(at + first, at + first + x.shape[0])
                lse[rows, h * group:(h + 1) * group] = torch.logsumexp(s, -1)
                out[rows, h * group:(h + 1) * group] = torch.einsum("ngk,kd->ngd", torch.softmax(s, -1), v)
        at += new
    return [out, lse] if case["lse"] else out
