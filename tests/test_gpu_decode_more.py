"""The decode operators on the GPU, further calls: batches whose partial sums are numbered by row or by token."""
import pytest
import torch

import filtered_int8_ann_b200 as st
from test_gpu_decode import check_attend, make_attend

pytestmark = pytest.mark.gpu


def widen(table, width):
    return [row + [-9] * (width - len(row)) for row in table]


@pytest.mark.parametrize("lens,qs,heads,group", [
    ([1300, 40, 900, 2000, 700], [1, 40, 8, 3, 50], 2, 4),     # numbered by row
    ([1300] + [60] * 19, [33] + [1] * 19, 1, 1),               # by token: few of the columns that the rows may have
    ([1300, 600, 1], [1, 1, 1], 2, 3)])
def test_attend_partial_sums(lens, qs, heads, group):
    """Stretches joined, with tokens behind the last row's and bounds above the rows' own."""
    q, codes, scales, table, start, lens = make_attend(50, lens, qs, heads, group, 64, 16, torch.float16)
    for spare in (0, 70):
        more = torch.cat([q, torch.zeros(spare, *q.shape[1:], dtype=q.dtype)])
        check_attend(more, codes, scales, table, start, lens)
        check_attend(more, codes, scales, table, start, lens, max_q=max(qs) + 5)


def test_attend_long_stretches_beside_prompts():
    """Rows that might be long, so many that their partial sums take longer stretches than 1024 tokens."""
    lens, qs = [2100, 70, 4500, 1030] + [20] * 60, [2, 40, 1, 3] + [1] * 60
    q, codes, scales, table, start, lens = make_attend(51, lens, qs, 8, 4, 128, 16, torch.bfloat16)
    for width in (4096, 8192):  # 65536 tokens: stretches of 2048; 131072: of 4096
        check_attend(q, codes, scales, widen(table, width), start, lens, max_len=16 * width)


@pytest.mark.parametrize("qs", [[1], [1, 1], [3, 90, 1]])
def test_attend_output_beside_the_queries(qs):
    """Output and queries as slices of one array: heads beside heads, every other head; further over is refused."""
    q, codes, scales, table, start, lens = make_attend(52, [2000 + m for m in qs], qs, 2, 4, 64, 16, torch.bfloat16)
    cache = st.KvCache(codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda())
    args = [torch.tensor(x, dtype=torch.int32).cuda() for x in (table, start, lens)] + [max(qs)]
    want = st.st_kv_attend(cache, q.cuda(), *args)
    for a, b in ((slice(0, 8), slice(8, 16)), (slice(0, 16, 2), slice(1, 16, 2))):
        hold = torch.zeros(q.shape[0], 16, 64, dtype=q.dtype, device="cuda")
        hold[:, a] = q.cuda()
        got = st.st_kv_attend(cache, hold[:, a], *args, out=hold[:, b])
        assert torch.equal(got, want) and torch.equal(hold[:, a], q.cuda())
    with pytest.raises(st.StError) as e:
        st.st_kv_attend(cache, hold[:, :8], *args, out=hold[:, 4:12])
    assert e.value.status == st.ST_ERR_INVALID_ARG


def test_reorder_outputs_beside_the_parents():
    x = torch.arange(24, dtype=torch.int32, device="cuda").view(2, 3, 4)
    beside = torch.zeros(30, dtype=torch.int32, device="cuda")
    got = st.st_beam_reorder([x], beside[24:].view(2, 3), out=[beside[:24].view(2, 3, 4)])
    assert torch.equal(got[0], x[:, :1].expand(2, 3, 4))
    with pytest.raises(st.StError) as e:
        st.st_beam_reorder([x], beside[:6].view(2, 3), out=[beside[:24].view(2, 3, 4)])
    assert e.value.status == st.ST_ERR_INVALID_ARG


def test_rows_not_served_are_planned_again():
    """The pool runs out in a step, a row ends, and the others are planned again: what the cache then holds is what a
    larger pool has (the prompt of each pair of rows is shared, so that blocks are replaced too)."""
    S, H, D, R, width = 16, 2, 64, 6, 4
    g = torch.Generator().manual_seed(60)
    i32 = dict(dtype=torch.int32, device="cuda")
    prompt = torch.randn(3 * 20, 2, H, D, generator=g).half().cuda()
    step = torch.randn(R, 2, H, D, generator=g).half().cuda()
    outs = []
    for blocks in (40, 8):  # 6 blocks hold the prompts; a step needs one block for each row
        cache = st.KvCache.empty(blocks, H, S, D)
        table, have = torch.full((R, width), -1, **i32), torch.zeros(R, **i32)
        slots, sources, start, lens, report = st.st_kv_plan(table, have, torch.tensor([20, 0] * 3, **i32), blocks, S, 60)
        assert report[2:].tolist() == [0, 0]
        st.st_kv_append(cache, prompt[:, 0], prompt[:, 1], slots, sources)
        table, have = table[::2].repeat_interleave(2, 0).contiguous(), lens[::2].repeat_interleave(2).contiguous()
        add, left, plans = torch.ones(R, **i32), torch.arange(R, device="cuda"), 0
        while True:
            slots, sources, start, lens, report = st.st_kv_plan(table, have, add, blocks, S, len(left))
            st.st_kv_append(cache, step[left, 0], step[left, 1], slots, sources)
            plans += 1
            unserved = lens < 0
            have, add = torch.where(unserved, have, lens), torch.where(unserved, add, 0)
            left = unserved.nonzero()[:, 0]
            if not len(left):
                break
            assert plans < 4 and int(report[2]) == len(left)
            if plans == 1:
                have[4:], add[4:] = 0, 0  # the last pair ends
                left = left[left < 4]
        assert plans == (1 if blocks == 40 else 2)
        assert have[:4].tolist() == [21] * 4 and len({int(table[r, 1]) for r in range(4)}) == 4
        q = torch.randn(4, 2 * H, D, generator=torch.Generator().manual_seed(61)).half().cuda()
        outs.append(st.st_kv_attend(cache, q, table[:4].contiguous(), torch.arange(5, **i32), have[:4].contiguous(), 1))
    assert torch.equal(*outs) and st.st_decode_check() == st.ST_OK


@pytest.mark.parametrize("queries", [1, 3, 40, 300])
@pytest.mark.parametrize("kind,power", [(kind, power) for kind in ("few", "most", "late", "near") for power in (10, 17, 24, 26, 40, 90)
                                        if kind != "near" or power <= 26])
def test_attend_scores_of_any_size(kind, power, queries):
    """Every score is a multiple of 2^power, so that the softmax is the mean over the tokens of the largest: `few` (three
    of 100 among 50s), `most` (the other way around, scores below zero), `late` (0 behind a long first part of large
    negative scores), `near` (as late, but 32 instead of 0, by a part of the query that fp16 holds up to 2^26).
    Tolerance: the output's half step, 2^-11 for the weights, 2^-20 for sums."""
    S, H, D, n = 16, 1, 64, 1600
    g = torch.Generator().manual_seed(power)
    blocks = n // S
    codes = [torch.zeros(blocks, H, S, D, dtype=torch.int8), torch.randint(-127, 128, (blocks, H, S, D), generator=g, dtype=torch.int8)]
    level = torch.full((n,), 0 if kind in ("late", "near") else 50)
    if kind in ("late", "near"):
        level[:700] = -100
    else:
        level[[7, 800, 1290]] = 100
    codes[0][..., 3] = level.view(blocks, H, S).to(torch.int8)
    scales = [torch.full((blocks, H), 0.5), torch.full((blocks, H), 2.0 ** -6)]
    q = torch.zeros(queries, 2, D)
    q[..., 3] = 2.0 ** power * (-1 if kind == "most" else 1)
    if kind == "near":
        codes[0].view(n, D)[700:, 5] = 8
        q[..., 5] = 8.0
    best = level == {"few": 100, "most": 50}.get(kind, 0)
    v = codes[1].view(n, D).double() * 2.0 ** -6
    got = st.st_kv_attend(st.KvCache(*(x.cuda() for x in codes), *(x.cuda() for x in scales)), q.bfloat16().cuda(),
                          torch.arange(blocks, dtype=torch.int32).view(1, -1).cuda(), torch.tensor([0, queries], dtype=torch.int32).cuda(),
                          torch.tensor([n], dtype=torch.int32).cuda(), queries, scale=1.0).cpu().double()
    for i in range(queries):
        seen = best & (torch.arange(n) <= n - queries + i)
        want, mass = v[seen].mean(0), v[seen].abs().mean(0)
        assert bool(((got[i] - want).abs() <= want.abs() * 2.0 ** -8 + mass * (2.0 ** -11 + 2.0 ** -20) * (1 + 2.0 ** -8)).all())


@pytest.mark.parametrize("queries", [1, 3, 40, 300])
def test_attend_scores_beyond_fp32(queries):
    """Above its range they give NaN, below it they count as not seen."""
    S, D, n = 16, 64, 1600
    codes = [torch.zeros(n // S, 1, S, D, dtype=torch.int8) for _ in range(2)]
    codes[0].view(n, D)[700:900, 3] = 100
    codes[1][:] = 64
    codes[1].view(n, D)[700:900] = -64
    scales = [torch.ones(n // S, 1), torch.full((n // S, 1), 2.0 ** -6)]
    cache = st.KvCache(*(x.cuda() for x in codes), *(x.cuda() for x in scales))
    i32 = dict(dtype=torch.int32, device="cuda")
    for sign in (1, -1):
        q = torch.zeros(queries, 2, D, dtype=torch.bfloat16, device="cuda")
        q[..., 3] = sign * 2.0 ** 125
        got = st.st_kv_attend(cache, q, torch.arange(n // S, **i32).view(1, -1), torch.tensor([0, queries], **i32), torch.tensor([n], **i32), queries, scale=1.0)
        assert bool(got.isnan().all() if sign > 0 else (got == 1).all())
        alone = st.st_kv_attend(cache, q, torch.arange(44, 55, **i32).view(1, -1), torch.tensor([0, queries], **i32), torch.tensor([170], **i32), queries, scale=1.0)
        seen = slice(max(0, queries - 170), queries)  # (queries before see nothing)
        assert bool(alone[seen].isnan().all() if sign > 0 else (alone == 0).all())


@pytest.mark.parametrize("queries", [1, 2, 40, 300])
@pytest.mark.parametrize("D,S,lens,extra", [
    (64, 16, [9001], 0), (128, 128, [16391], 0), (64, 64, [40013], 0), (64, 32, [1023, 4097, 2560, 300], 0), (128, 16, [1025, 513, 7000], 0),
    (128, 64, [5000, 1024, 3073], 60000)])
@pytest.mark.parametrize("by", ["turns", "parts"])
def test_attend_counts_every_token_once(by, D, S, lens, extra, queries):
    """Equal scores: each dim holds the share of the tokens that are its own, by turns or one part of the row after the
    other. A token that is left out or taken twice moves its dim by 1 / tokens of the dim, which is above the
    tolerance: half a step of fp16 and of the weights (2^-11 each), 2^-20 for sums."""
    H, R = 2, len(lens)
    width = (max(lens) + extra) // S + 2
    pages = [-(-n // S) for n in lens]
    order = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(D + S)).int()
    table, codes, at = torch.full((R, width), -1, dtype=torch.int32), torch.zeros(sum(pages), H, S, D, dtype=torch.int8), 0
    owners = []
    for r, (n, p) in enumerate(zip(lens, pages)):
        j = torch.arange(n)
        own = j % D if by == "turns" else torch.clamp(j // -(-n // D), max=D - 1)
        row = torch.zeros(p * S, D, dtype=torch.int8)
        row[j, own] = 100
        table[r, :p] = order[at:at + p]
        codes[order[at:at + p].long()] = row.view(p, 1, S, D).expand(p, H, S, D)
        at += p
        owners.append(own)
    ones = torch.full((sum(pages), H), 2.0 ** -5, device="cuda")
    cache = st.KvCache(torch.randint(-127, 128, codes.shape, dtype=torch.int8, device="cuda"), codes.cuda(), ones, ones.clone())
    start = torch.arange(R + 1, dtype=torch.int32) * queries
    q = torch.zeros(R * queries, 2 * H, D, dtype=torch.float16, device="cuda")
    got = st.st_kv_attend(cache, q, table.cuda(), start.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), queries,
                          max_len=max(lens) + extra).cpu().double()
    for r, n in enumerate(lens):
        for i in {0, queries // 2, queries - 1}:
            seen = n - queries + i + 1
            want = torch.bincount(owners[r][:max(0, seen)], minlength=D).double() / max(1, seen) * 100 / 32
            off = (got[r * queries + i] - want).abs()
            assert bool((off <= want * (2.0 ** -10 + 2.0 ** -19)).all()), (r, i, float((off / want).max()))
