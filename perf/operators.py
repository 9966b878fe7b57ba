"""The operators of one beam decode step over an int8 paged cache: cases, inputs, plain forms and 64-bit values.

plan     block tables and slot maps of the rows from their lengths, with a new page for a shared last page
append   new keys and values into the int8 cache, one scale per page and head
attend   attention of one or more query tokens per row over that cache
select   the best (beam, token) pairs of each request
reorder  the states of the chosen beams
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # a step of sixteen requests of four beams, a few thousand tokens each: the tables' smallest ordinary call
        {"name": "plan beams", "op": "plan", "rows": 64, "beams": 4, "len": 2000, "add": 1, "block": 16},
        # a scheduler's largest call: a thousand prompts of up to a thousand tokens join at once
        {"name": "plan prompts", "op": "plan", "rows": 1024, "beams": 1, "len": 0, "add": 1000, "block": 32},
        # one token for each of 256 rows
        {"name": "append step", "op": "append", "rows": 256, "add": 1, "kv_heads": 8, "dim": 128, "block": 16, "dtype": "bf16"},
        # prompts of two thousand tokens
        {"name": "append prompts", "op": "append", "rows": 7, "add": 2049, "kv_heads": 8, "dim": 128, "block": 64, "dtype": "f16"},
        # a few short rows: latency
        {"name": "attend short", "op": "attend", "rows": 8, "kv_heads": 4, "group": 2, "dim": 64, "block": 16, "len": 500, "ragged": True, "q": 1, "dtype": "f16"},
        # a full batch of long rows of uneven lengths: the serving load
        {"name": "attend batch", "op": "attend", "rows": 64, "kv_heads": 8, "group": 4, "dim": 128, "block": 32, "len": 16384, "ragged": True, "q": 1, "dtype": "bf16"},
        # one user with a long history: the work is split along the cache
        {"name": "attend one", "op": "attend", "rows": 1, "kv_heads": 8, "group": 8, "dim": 128, "block": 64, "len": 100003, "ragged": False, "q": 1, "dtype": "bf16"},
        # chunks of long prompts: products bound
        {"name": "attend prompts", "op": "attend", "rows": 4, "kv_heads": 8, "group": 4, "dim": 128, "block": 64, "len": 8192, "ragged": True, "q": 2048, "dtype": "bf16"},
        # codes of items: a small vocabulary of which each beam may take only some entries
        {"name": "select codes", "op": "select", "requests": 8, "beams": 16, "vocab": 1021, "keep": 16, "masked": True, "finished": False, "dtype": "f32"},
        # words: a large vocabulary, twice the beams kept, some of them finished
        {"name": "select words", "op": "select", "requests": 32, "beams": 32, "vocab": 100003, "keep": 64, "masked": False, "finished": True, "dtype": "bf16"},
        # the block tables and token histories of paged beams
        {"name": "reorder tables", "op": "reorder", "requests": 16, "beams": 8, "arrays": 2, "width": 511, "dtype": "i32"},
        # dense states of four layers
        {"name": "reorder states", "op": "reorder", "requests": 16, "beams": 8, "arrays": 4, "width": 262144, "dtype": "bf16"},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "select", "reorder"])
    block = rng.choice([16, 32, 64, 128])
    if op == "plan":
        beams = rng.choice([1, 1, 2, 4, 5, 8])
        rows = beams * max(1, _log(rng, 1, 1024) // beams)
        if rng.random() < 0.5:
            return {"op": op, "rows": rows, "beams": beams, "len": _log(rng, 1, 8192), "add": rng.randint(1, 4), "block": block}
        return {"op": op, "rows": rows, "beams": 1, "len": rng.choice([0, _log(rng, 1, 500)]), "add": _log(rng, 2, 1000), "block": block}
    if op == "append":
        kv_heads, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
        rows = _log(rng, 1, 512)
        add = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 14336 * 1024 // (rows * kv_heads * dim)))
        return {"op": op, "rows": rows, "add": add, "kv_heads": kv_heads, "dim": dim, "block": block, "dtype": rng.choice(["bf16", "f16"])}
    if op == "attend":
        kv_heads, dim, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        q = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 16, 2048)])
        length = _log(rng, max(q, 8), 65536 if q <= 8 else 8192)
        most = 64 * 16384 * 8 * 128 // (length * kv_heads * dim)
        most = min(most, 4 * 2048 * 32 * 8192 // (q * group * kv_heads * length))
        rows = _log(rng, 1, max(1, min(256, most)))
        return {"op": op, "rows": rows, "kv_heads": kv_heads, "group": group, "dim": dim, "block": block, "len": length, "ragged": rng.random() < 0.7, "q": q, "dtype": rng.choice(["bf16", "f16"])}
    if op == "select":
        beams, vocab = _log(rng, 1, 64), _log(rng, 64, 200000)
        requests = _log(rng, 1, max(1, min(64, 32 * 32 * 100003 // (beams * vocab))))
        return {"op": op, "requests": requests, "beams": beams, "vocab": vocab, "keep": beams * rng.choice([1, 2]), "masked": rng.random() < 0.3, "finished": rng.random() < 0.3, "dtype": rng.choice(["bf16", "f16", "f32"])}
    beams, arrays = rng.randint(1, 16), rng.randint(1, 6)
    requests = _log(rng, 1, 64)
    return {"op": op, "requests": requests, "beams": beams, "arrays": arrays, "width": _log(rng, 5, max(6, min(500000, 16 * 8 * 4 * 262144 // (2 * requests * beams * arrays)))), "dtype": rng.choice(["bf16", "i32", "f32", "i8"])}


# ---------------------------------------------------------------- sizes --
def _lens(c):
    """Stored tokens of each row (attend), new ones included; uneven ones go down to a quarter, one row has none."""
    n, full = c["rows"], c["len"]
    if not c["ragged"]:
        return [full] * n
    lens = [max(1, round(full * (1 - 0.75 * i / max(1, n - 1)))) for i in range(n)]
    if n >= 4:
        lens[-1] = 0
        lens[-2] = 1
    return lens


def _queries(c):
    """Query tokens of each row: all of them in an even batch, else 1 to q, no more than the row holds."""
    return [max(1, min(c["q"], n)) if not c["ragged"] else max(1, min(1 + (7 * c["q"] // 8 + 977 * i) % c["q"], n)) for i, n in enumerate(_lens(c))]


def _plan_rows(c):
    """(have, add) of each row; the beams of one request are alike."""
    groups = c["rows"] // c["beams"]
    have, add = [], []
    for g in range(groups):
        n = round(c["len"] * (1 - 0.75 * g / max(1, groups - 1)))
        m = c["add"] if c["beams"] > 1 or c["add"] == 1 else 1 + (c["add"] // 2 + 389 * g) % c["add"]
        have += [n] * c["beams"]
        add += [m] * c["beams"]
    return have, add


def _ceil(a, b):
    return -(-a // b)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# -------------------------------------------------------------- prepare --
def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "attend": _prepare_attend, "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]](case, seed)


def _prepare_plan(c, seed):
    r, g = random.Random(seed), _gen(seed)
    have, add = _plan_rows(c)
    order = list(range(c["rows"] // c["beams"]))
    r.shuffle(order)  # which request has which length
    bs, beams = c["block"], c["beams"]
    width = _ceil(max(h + a for h, a in zip(have, add)), bs)
    rows, h2, a2, count = [], [], [], 0
    for at, k in enumerate(order):
        n = _ceil(have[k * beams], bs)
        base = list(range(count, count + n))
        count += n
        for b in range(beams):
            mine = list(base)
            if at % 2 and b and n:  # every other request: its beams have a last page of their own already
                mine[-1] = count
                count += 1
            rows.append(mine)
        h2 += have[k * beams:(k + 1) * beams]
        a2 += add[k * beams:(k + 1) * beams]
    most = sum(_ceil(h + a, bs) - _ceil(h, bs) + 1 for h, a in zip(h2, a2))
    blocks = count + most + most // 8 + 8
    perm = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    flat = torch.full((c["rows"], width), -1, dtype=torch.int64)
    for i, m in enumerate(rows):
        flat[i, :len(m)] = torch.tensor(m, dtype=torch.int64)
    flat = flat.cuda()
    table = torch.where(flat >= 0, perm[flat.clamp(min=0)], flat.int()).contiguous()
    return {"op": "plan", "table": table, "have": torch.tensor(h2, dtype=torch.int32).cuda(), "add": torch.tensor(a2, dtype=torch.int32).cuda(), "blocks": blocks, "block": bs, "tokens": sum(a2) + 3}


def _prepare_append(c, seed):
    r, g = random.Random(seed), _gen(seed)
    bs, heads, dim, n = c["block"], c["kv_heads"], c["dim"], c["rows"]
    offs = [(37 * i + 5) % bs for i in range(n)]  # tokens already in each row's first page
    r.shuffle(offs)
    pages = [_ceil(o + c["add"], bs) for o in offs]
    spare = _ceil(n, 4)
    blocks = sum(pages) + spare
    perm = torch.randperm(blocks, generator=g, device="cuda")
    slots, sources, at = [], [], 0
    for i, (o, p) in enumerate(zip(offs, pages)):
        pos = torch.arange(o, o + c["add"])
        page = at + pos // bs
        slots.append(page * bs + pos % bs)
        sources.append(torch.where(pos < bs, sum(pages) + i // 4, page) if i % 4 == 3 and o else page)  # a last page shared before: its tokens come from another
        at += p
    slots, sources = torch.cat(slots).cuda(), torch.cat(sources).cuda()
    slots = perm[slots // bs] * bs + slots % bs
    kv = torch.randn(2, blocks, heads, bs, dim, generator=g, device="cuda", dtype=torch.float16).mul_(40).clamp_(-127, 127).to(torch.int8)
    scale = (2 + 2 * torch.rand(2, blocks, heads, generator=g, device="cuda")) / 127
    new = torch.randn(n * c["add"], 2, heads, dim, generator=g, device="cuda").to(DTYPES[c["dtype"]])
    return {"op": "append", "kv": kv, "scale": scale, "new": new, "slots": slots, "sources": perm[sources].int()}


def _prepare_attend(c, seed):
    r, g = random.Random(seed), _gen(seed)
    bs, heads, dim, n = c["block"], c["kv_heads"], c["dim"], c["rows"]
    rows = list(zip(_lens(c), _queries(c)))
    r.shuffle(rows)
    lens, qs = [x for x, _ in rows], [x for _, x in rows]
    start = [0]
    for x in qs:
        start.append(start[-1] + x)
    width = _ceil(c["len"], bs)
    pages = [_ceil(x, bs) for x in lens]
    blocks = sum(pages) + 4
    perm = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    table = torch.zeros(n, width, dtype=torch.int32, device="cuda")
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = perm[at:at + p]
        at += p
    kv = torch.randn(2, blocks, heads, bs, dim, generator=g, device="cuda", dtype=torch.float16).mul_(40).clamp_(-127, 127).to(torch.int8)
    scale = (2 + 2 * torch.rand(2, blocks, heads, generator=g, device="cuda")) / 127
    q = (2 * torch.randn(start[-1], heads * c["group"], dim, generator=g, device="cuda")).to(DTYPES[c["dtype"]])
    return {"op": "attend", "kv": kv, "scale": scale, "q": q, "table": table, "start": torch.tensor(start, dtype=torch.int32).cuda(), "lens": torch.tensor(lens, dtype=torch.int32).cuda(),
            "most": max(qs), "len": c["len"], "factor": dim ** -0.5}


def _prepare_select(c, seed):
    g = _gen(seed)
    b, k, v = c["requests"], c["beams"], c["vocab"]
    x = (3 * torch.randn(b, k, v, generator=g, device="cuda")).to(DTYPES[c["dtype"]])
    scores = -20 * torch.rand(b, k, generator=g, device="cuda")
    s = {"op": "select", "logits": x, "scores": scores, "keep": c["keep"], "end": v // 3, "allow": None, "finished": None}
    if c["masked"]:  # a bit per token
        words = torch.randint(-2**31, 2**31 - 1, (2, b, k, _ceil(v, 32)), generator=g, device="cuda", dtype=torch.int64).int()
        s["allow"] = words[0] & words[1]
    if c["finished"]:
        s["finished"] = torch.rand(b, k, generator=g, device="cuda") < 0.25
    return s


def _prepare_reorder(c, seed):
    g = _gen(seed)
    b, k = c["requests"], c["beams"]
    shape = (b, k, c["width"])
    if c["dtype"] in DTYPES:
        states = [torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[c["dtype"]]) for _ in range(c["arrays"])]
    else:
        kind = {"i32": torch.int32, "i8": torch.int8}[c["dtype"]]
        states = [torch.randint(-120, 120, shape, generator=g, device="cuda", dtype=kind) for _ in range(c["arrays"])]
    return {"op": "reorder", "states": states, "parents": torch.randint(0, k, (b, k), generator=g, device="cuda", dtype=torch.int32)}


# ------------------------------------------------------------------ run --
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_plan(s):
    import filtered_int8_ann_b200 as st
    slots, sources, start, lens, report = st.st_kv_plan(s["table"], s["have"], s["add"], s["blocks"], s["block"], s["tokens"])
    return {"table": s["table"], "slots": slots, "sources": sources, "start": start, "lens": lens, "report": report}


def _plain_plan(s):
    table, have, add, bs, blocks = s["table"], s["have"].long(), s["add"].long(), s["block"], s["blocks"]
    rows, width = table.shape
    col = torch.arange(width, device="cuda")
    used = (have + bs - 1) // bs
    stored = torch.where(col < used[:, None], table.long(), blocks)
    refs = torch.zeros(blocks + 1, dtype=torch.int64, device="cuda").scatter_add_(0, stored.flatten(), torch.ones_like(stored).flatten())[:blocks]
    tail = table.gather(1, (used - 1).clamp(min=0)[:, None])[:, 0].long().clamp(min=0)
    copied = ((have % bs > 0) & (add > 0) & (refs[tail] > 1)).long()
    need = (have + add + bs - 1) // bs - used + copied
    end = need.cumsum(0)
    free = refs == 0
    count = free.sum()
    rank = free.cumsum(0) - 1
    pages = torch.zeros(blocks + 1, dtype=torch.int64, device="cuda").scatter_(0, torch.where(free, rank, blocks), torch.arange(blocks, device="cuda"))
    served = (need == 0) | (end <= count)
    at = col - (used - copied)[:, None]
    new = (at >= 0) & (at < need[:, None]) & served[:, None]
    table.copy_(torch.where(new, pages[((end - need)[:, None] + at).clamp(0, blocks)], table.long()))
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), add.cumsum(0)])
    t = torch.arange(s["tokens"], device="cuda")
    row = torch.searchsorted(start[1:], t, right=True).clamp(max=rows - 1)
    real = (t < start[-1]) & served[row]
    pos = have[row] + t - start[row]
    page = table[row, (pos // bs).clamp(max=width - 1)].long()
    slots = torch.where(real, page * bs + pos % bs, -1)
    first = (copied[row] > 0) & (pos // bs == used[row] - 1)
    sources = torch.where(real, torch.where(first, tail[row], page), -1).int()
    lens = torch.where(served, have + add, -1).int()
    report = torch.stack([need.sum(), count, (~served).sum(), torch.zeros_like(count)]).int()
    return {"table": table, "slots": slots, "sources": sources, "start": start.int(), "lens": lens, "report": report}


def _values(s):
    """The cache as the numbers that it stands for, in the type of the new keys and values."""
    out = torch.empty(s["kv"].shape, dtype=s["new"].dtype, device="cuda")
    return torch.mul(s["kv"], s["scale"][..., None, None], out=out)


def _own_append(s):
    import filtered_int8_ann_b200 as st
    kv, scale, new = s["kv"], s["scale"], s["new"]
    st.st_kv_append(st.KvCache(kv[0], kv[1], scale[0], scale[1]), new[:, 0], new[:, 1], s["slots"], s["sources"])
    return _values(s)


def _plain_append(s):
    kv, scale, slots, sources = s["kv"], s["scale"], s["slots"], s["sources"].long()
    _, blocks, heads, bs, dim = kv.shape
    page, off = slots // bs, slots % bs
    first = torch.ones_like(page, dtype=torch.bool)  # first token of a run inside one page
    first[1:] = slots[1:] != slots[:-1] + 1
    first |= off == 0
    at = first.nonzero()[:, 0]  # first token of each run
    run_of = first.cumsum(0) - 1
    x = s["new"].float().transpose(0, 1)  # [2, T, heads, dim]
    peak = x.abs().amax(-1)  # [2, T, heads]
    amax = torch.zeros(2, at.numel(), heads, device="cuda").scatter_reduce_(1, run_of[None, :, None].expand_as(peak), peak, "amax")
    old, to, of = off[at], page[at], sources[at]  # tokens that stand in the run's page already, its page, and the page to take them from
    before = torch.where(old[None, :, None] > 0, scale[:, of], 0.0)
    after = torch.maximum(before, amax / 127)
    after = torch.where(after > 2.0**-100, after, 0.0)
    ratio = torch.where(after > 0, before / after, 0.0)
    turn = torch.where(after > 0, 1 / after, 0.0)
    stay = torch.arange(bs, device="cuda") < old[:, None]  # [runs, bs]
    moved = torch.round(kv[:, of] * ratio[..., None, None])
    kv[:, to] = torch.where(stay[None, :, None, :, None], moved, kv[:, to].float()).to(torch.int8)
    scale[:, to] = after
    codes = torch.round(x * turn[:, run_of][..., None]).clamp(-127, 127).to(torch.int8)
    kv[0, page, :, off] = codes[0]
    kv[1, page, :, off] = codes[1]
    return _values(s)


def _own_attend(s):
    import filtered_int8_ann_b200 as st
    kv, scale = s["kv"], s["scale"]
    return st.st_kv_attend(st.KvCache(kv[0], kv[1], scale[0], scale[1]), s["q"], s["table"], s["start"], s["lens"], s["most"], max_len=s["len"], scale=s["factor"])


def _plain_attend(s):
    kv, scale, q, table, lens, most = s["kv"], s["scale"], s["q"], s["table"].long(), s["lens"].long(), s["most"]
    start = s["start"].long()
    rows, width = table.shape
    _, _, heads, bs, dim = kv.shape
    group = q.shape[1] // heads
    t = torch.arange(q.shape[0], device="cuda")
    row = torch.searchsorted(start[1:], t, right=True)
    j = t - start[row]
    padded = torch.zeros(rows, most, heads * group, dim, device="cuda")
    padded[row, j] = q.float()
    padded = padded.view(rows, most, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(rows, heads, group * most, dim)

    def dense(i):
        x = kv[i][table].float().mul_(scale[i][table][..., None, None])  # [rows, width, heads, bs, dim]
        return x.transpose(1, 2).reshape(rows, heads, width * bs, dim)

    w = (padded * s["factor"]) @ dense(0).transpose(-1, -2)
    count = start[1:] - start[:-1]
    last = (lens - count)[:, None] + torch.arange(most, device="cuda")  # the last position that query j sees
    sees = torch.arange(width * bs, device="cuda") <= last[..., None]
    sees &= torch.arange(width * bs, device="cuda") < lens[:, None, None]
    w = w.view(rows, heads, group, most, width * bs)
    w.masked_fill_(~sees[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    o = w.view(rows, heads, group * most, width * bs) @ dense(1)
    o = o.view(rows, heads, group, most, dim) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(rows, most, heads * group, dim)
    return o[row, j].to(q.dtype)


def _own_select(s):
    import filtered_int8_ann_b200 as st
    scores, parents, tokens, finished = st.st_beam_select(s["logits"], s["scores"], s["keep"], allow=s["allow"], finished=s["finished"], end_token=s["end"])
    out = {"scores": scores, "parents": parents, "tokens": tokens}
    return out if finished is None else {**out, "finished": finished}


def _plain_select(s):
    x, base, n = s["logits"].double(), s["scores"].double(), s["keep"]
    b, k, v = x.shape
    if s["allow"] is not None:
        bit = torch.arange(v, device="cuda")
        x = torch.where((s["allow"][..., bit // 32] >> (bit % 32).int()) & 1 > 0, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    x = x - (top + (x - top).exp().sum(-1, keepdim=True).log()) + base[..., None]
    if s["finished"] is not None:
        done = torch.full_like(x, -math.inf)
        done[..., s["end"]] = base
        x = torch.where(s["finished"][..., None], done, x)
    x = x.nan_to_num(nan=-math.inf, neginf=-math.inf).view(b, k * v)
    n_here = min(n, k * v)
    border = x.topk(n_here, -1).values[:, -1:]
    more, like = x > border, x == border
    like &= like.cumsum(-1) <= n_here - more.sum(-1, keepdim=True)
    at = (more | like).nonzero()[:, 1].view(b, n_here)  # in the order of their index
    value = x.gather(1, at)
    order = value.sort(dim=-1, descending=True, stable=True).indices
    value, at = value.gather(1, order), at.gather(1, order)
    none = value == -math.inf
    parents, tokens = torch.where(none, -1, at // v).int(), torch.where(none, -1, at % v).int()
    fill = lambda a, with_: torch.cat([a, torch.full((b, n - n_here), with_, dtype=a.dtype, device="cuda")], 1)  # noqa: E731
    out = {"scores": fill(value.float(), -math.inf), "parents": fill(parents, -1), "tokens": fill(tokens, -1)}
    if s["finished"] is not None:
        old = s["finished"].gather(1, out["parents"].clamp(min=0).long())
        out["finished"] = (out["parents"] >= 0) & (old | (out["tokens"] == s["end"]))
    return out


def _own_reorder(s):
    import filtered_int8_ann_b200 as st
    return st.st_beam_reorder(s["states"], s["parents"])


def _plain_reorder(s):
    b, k = s["parents"].shape
    at = s["parents"].long() + k * torch.arange(b, device="cuda")[:, None]
    return [x.flatten(0, 1)[at] for x in s["states"]]


_own = {"plan": _own_plan, "append": _own_append, "attend": _own_attend, "select": _own_select, "reorder": _own_reorder}
_plain = {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend, "select": _plain_select, "reorder": _plain_reorder}


# ----------------------------------------------------------------- work --
def work(case):
    c = case
    if c["op"] == "plan":
        have, add = _plan_rows(c)
        read = sum(4 * _ceil(h, c["block"]) for h in have) + 8 * len(have)
        written = sum(4 * (_ceil(h + a, c["block"]) - _ceil(h, c["block"])) for h, a in zip(have, add)) + 8 * len(have) + 12 * sum(add)
        return {"bytes": read + written, "flops": 0}
    if c["op"] == "append":  # new values read, their codes written
        n = 2 * c["rows"] * c["add"] * c["kv_heads"] * c["dim"]
        return {"bytes": 3 * n + 12 * c["rows"] * c["add"], "flops": 2 * n}
    if c["op"] == "attend":
        lens, qs = _lens(c), _queries(c)
        heads = c["kv_heads"] * c["group"]
        cache = sum(2 * c["kv_heads"] * (n * c["dim"] + 4 * _ceil(n, c["block"])) + 4 * _ceil(n, c["block"]) for n in lens)
        pairs = sum(q * n - q * (q - 1) // 2 for n, q in zip(lens, qs) if n)
        return {"bytes": cache + 4 * sum(qs) * heads * c["dim"], "flops": 4 * pairs * heads * c["dim"]}
    if c["op"] == "select":
        rows = c["requests"] * c["beams"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": rows * (c["vocab"] * size + (c["vocab"] / 8 if c["masked"] else 0) + 4) + 12 * c["requests"] * c["keep"], "flops": 3 * rows * c["vocab"]}
    size = {"bf16": 2, "i32": 4, "f32": 4, "i8": 1}[c["dtype"]]
    n = c["requests"] * c["beams"]
    return {"bytes": 2 * size * n * c["arrays"] * c["width"] + 4 * n, "flops": 0}


# ---------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": lambda s: None, "append": _exact_append, "attend": _exact_attend, "select": _exact_select, "reorder": _exact_reorder}[s["op"]](s)


def _exact_append(s):
    kv, scale, bs = s["kv"], s["scale"].double(), s["kv"].shape[3]
    slots, sources = s["slots"].tolist(), s["sources"].tolist()
    value = kv.double() * scale[..., None, None]
    at = 0
    while at < len(slots):
        page, off = divmod(slots[at], bs)
        end = at + 1
        while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] % bs:
            end += 1
        n = end - at
        x = s["new"][at:end].double().permute(1, 2, 0, 3)  # [2, heads, n, dim]
        peak = x.abs().amax((-1, -2)) / 127
        if off:
            peak = torch.maximum(peak, scale[:, sources[at]])
        step = peak[..., None, None]
        inside = torch.arange(bs, device="cuda")[:, None]
        if off:
            old = (value[:, sources[at]] / step).round() * step
            value[:, page] = torch.where(inside < off, old, kv[:, page].double() * step)
        else:
            value[:, page] = kv[:, page].double() * step
        value[:, page, :, off:off + n] = (x / step).round().clamp(-127, 127) * step
        at = end
    return value


def _exact_attend(s):
    kv, scale, q = s["kv"], s["scale"].double(), s["q"].double()
    heads, bs, dim = kv.shape[2:]
    group = q.shape[1] // heads
    start, lens, table = s["start"].tolist(), s["lens"].tolist(), s["table"].long()
    out = torch.zeros_like(q)
    for r, n in enumerate(lens):
        if not n:
            continue
        pages = table[r, :_ceil(n, bs)]
        m = start[r + 1] - start[r]
        hidden = torch.arange(n, device="cuda")[None, :] > torch.arange(n - m, n, device="cuda")[:, None]
        for h in range(heads):
            k, v = ((kv[i, pages, h].double() * scale[i, pages, h][:, None, None]).reshape(-1, dim)[:n] for i in (0, 1))
            for g in range(group):
                w = (q[start[r]:start[r + 1], h * group + g] @ k.T) * s["factor"]
                out[start[r]:start[r + 1], h * group + g] = torch.softmax(w.masked_fill(hidden, -math.inf), -1) @ v
    return out


def _exact_select(s):
    """The scores alone; which pairs they belong to are whole numbers."""
    x, base, n = s["logits"], s["scores"].double(), s["keep"]
    b, k, v = x.shape
    found = torch.full((b, n), -math.inf, dtype=torch.float64, device="cuda")
    for i in range(b):
        rows = []
        for j in range(k):
            if s["finished"] is not None and s["finished"][i, j]:
                rows.append(base[i, j].reshape(1))
                continue
            y = x[i, j].double()
            if s["allow"] is not None:
                words = s["allow"][i, j].long() & 0xFFFFFFFF
                y = y[((words[:, None] >> torch.arange(32, device="cuda")) & 1).flatten()[:v] > 0]
            if y.numel():
                rows.append((torch.log_softmax(y, 0) + base[i, j]).sort(descending=True).values[:n])
        if rows:
            best = torch.cat(rows).sort(descending=True).values[:n]
            found[i, :best.numel()] = best
    out = {"scores": found, "parents": None, "tokens": None}
    return out if s["finished"] is None else {**out, "finished": None}


def _exact_reorder(s):
    if not s["states"][0].is_floating_point():
        return None
    b, k = s["parents"].shape
    chosen = s["parents"].tolist()
    return [torch.stack([torch.stack([x[i, chosen[i][j]] for j in range(k)]) for i in range(b)]).double() if x.is_floating_point() else None for x in s["states"]]
