"""The decode operators on the GPU against their plain forms (decode_ref.py)."""
import math
import random

import numpy as np
import pytest
import torch

import decode_ref as ref
import filtered_int8_ann_b200 as st

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------- plan --
def run_plan(table, have, add, blocks, S, T):
    t = torch.tensor(table, dtype=torch.int32).cuda()
    out = st.st_kv_plan(t, torch.tensor(have, dtype=torch.int32).cuda(), torch.tensor(add, dtype=torch.int32).cuda(), blocks, S, T)
    torch.cuda.synchronize()
    return [t.tolist()] + [o.tolist() for o in out]


def check_plan(table, have, add, blocks, S, T, bad=False):
    got = run_plan(table, have, add, blocks, S, T)
    assert st.st_decode_check() == (st.ST_ERR_DEVICE if bad else st.ST_OK)
    want = ref.plan(table, have, add, blocks, S, T)
    for g, w, name in zip(got, want, ("table", "slots", "sources", "row_start", "lens", "report")):
        assert g == list(w), name
    return got


def random_rows(r, R, S, width, blocks, share):
    pool = list(range(blocks))
    r.shuffle(pool)
    table, have = [], []
    for i in range(R):
        if i and share and r.random() < share:  # a beam of the row before: some of its blocks
            h = r.randint(0, have[-1])
            table.append(list(table[-1]))
            have.append(h)
            continue
        h = min(width * S, r.choice([0, 1, S - 1, S, S + 1, r.randint(0, width * S)]))
        n = -(-h // S)
        if n > len(pool):
            h = n = 0
        table.append([pool.pop() for _ in range(n)] + [-7] * (width - n))
        have.append(h)
    return table, have


@pytest.mark.parametrize("seed", range(12))
def test_plan_random(seed):
    r = random.Random(seed)
    S = r.choice([16, 32, 64, 128])
    R, width = r.choice([1, 3, 31, 32, 33, 100, 260]), r.choice([1, 2, 5, 40])
    blocks = R * width + r.randint(1, 70)
    table, have = random_rows(r, R, S, width, blocks, r.choice([0, 0.5, 0.9]))
    add = [r.choice([0, 1, 1, 2, S, r.randint(0, 2 * S)]) for _ in range(R)]
    T = sum(add) + r.choice([0, 1, 33])
    check_plan(table, have, add, blocks, S, T)


def test_plan_pool_runs_out_in_order():
    S = 16
    table = [[0, -1, -1], [1, -1, -1], [2, -1, -1], [-1, -1, -1], [3, -1, -1]]
    # rows 1 and 3 want more than is left; row 2 and row 4 need none
    got = check_plan(table, [16, 16, 5, 0, 5], [16, 17, 3, 1, 4], 6, S, 41)
    assert got[4] == [32, -1, 8, -1, 9]
    assert got[5][2:] == [2, 0]


def test_plan_refuses_malformed_rows_and_marks_the_error_word():
    S = 16
    table = [[0, 99], [1, -3], [2, 3], [4, 5], [6, 7], [8, 9]]
    check_plan(table, [20, 20, -1, 16, 40, 16], [1, 1, 1, -2, 1, 30], 20, S, 40, bad=True)


def test_plan_without_room_for_the_tokens():
    check_plan([[0, -1], [1, -1], [2, -1]], [3, 3, 3], [2, 5, 1], 8, 16, 4)
    check_plan([[0, -1], [1, -1]], [3, 3], [0, 0], 8, 16, 0)


def test_plan_shared_tails_are_replaced_for_every_writer():
    S = 16
    table = [[0, 1, -1]] * 4 + [[0, 2, -1]] + [[3, 3, -1]]
    got = check_plan(table, [20, 20, 20, 20, 20, 20], [1, 1, 0, 13, 1, 1], 12, S, 20)
    new = [got[0][i][1] for i in (0, 1, 3)]
    assert len(set(new + [1])) == 4 and got[0][2] == [0, 1, -1] and got[0][4][1] == 2
    assert got[0][5][0] == 3 and got[0][5][1] != 3


@pytest.mark.parametrize("R,width,blocks", [(32768, 3, 100000), (7, 4000, 40000), (300, 20, 4194304)])
def test_plan_largest_sizes(R, width, blocks):
    r = random.Random(5)
    S = 16
    per = min(width - 1, blocks // R)
    have = [r.randint(0, per * S) for _ in range(R)]
    pages = iter(torch.randperm(blocks, generator=gen(1))[: R * per].tolist())
    table = [[next(pages) for _ in range(per)] + [-1] * (width - per) for _ in range(R)]
    add = [r.randint(0, 3) for _ in range(R)]
    check_plan(table, have, add, blocks, S, sum(add) + 5)


def test_plan_refuses_overlapping_arrays():
    i32 = dict(dtype=torch.int32, device="cuda")
    table, have, add = torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.ones(2, **i32)
    for kw in (dict(lens=have), dict(lens=add), dict(report=table.view(-1)[:4])):
        with pytest.raises(st.StError) as e:
            st.st_kv_plan(table, have, add, 9, 16, 2, **kw)
        assert e.value.status == st.ST_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        st.st_kv_plan(table, have, add, 9, 16, -1)


# ----------------------------------------------------------------- append --
def check_append(x, cache, slots, sources, bad=False, spread=False):
    """x: [T, 2, heads, D]"""
    want = [cache[0].numpy().copy(), cache[1].numpy().copy(), cache[2].numpy().copy(), cache[3].numpy().copy()]
    for i in range(2):
        ref.append(want[i], want[2 + i], x[:, i].float().numpy(), slots, sources)
    dev = [c.cuda() for c in cache]
    xs = x.cuda()
    k, v = xs[:, 0], xs[:, 1]
    if spread:  # heads and tokens far apart
        wide = torch.empty(x.shape[0], x.shape[2], 2, x.shape[3] + 8, dtype=x.dtype, device="cuda")
        wide[:, :, 0, :x.shape[3]] = k
        k = wide[:, :, 0, :x.shape[3]]
    st.st_kv_append(st.KvCache(*dev), k, v, torch.tensor(slots, dtype=torch.int64).cuda(),
                    None if sources is None else torch.tensor(sources, dtype=torch.int32).cuda())
    assert st.st_decode_check() == (st.ST_ERR_DEVICE if bad else st.ST_OK)
    for g, w, name in zip(dev, want, ("k", "v", "k_scale", "v_scale")):
        assert np.array_equal(g.cpu().numpy(), w), name


def new_cache(g, blocks, heads, S, D):
    return [torch.randint(-127, 128, (blocks, heads, S, D), generator=g, dtype=torch.int8) for _ in range(2)] + \
        [torch.rand(blocks, heads, generator=g) * 0.05 for _ in range(2)]


@pytest.mark.parametrize("S", [16, 32, 64, 128])
@pytest.mark.parametrize("D,heads,dtype", [(64, 3, torch.bfloat16), (128, 2, torch.float16), (128, 1, torch.bfloat16), (64, 1, torch.float16)])
def test_append_runs(S, D, heads, dtype):
    """Runs of every kind: whole blocks, inside one, over several, from a shared block, single tokens, skipped ones."""
    g = gen(S + D)
    blocks = 24
    cache = new_cache(g, blocks, heads, S, D)
    slots, sources = [], []

    def run(page, off, n, src=None):
        while n:
            m = min(n, S - off)
            slots.extend(page * S + off + i for i in range(m))
            sources.extend([page if src is None else src] * m)
            page, off, n, src = page + 1, 0, n - m, None

    run(0, 0, 3 * S + 1)
    run(5, S - 1, 2)
    run(8, 1, 1)
    slots += [-1, -1]
    sources += [-1, -1]
    run(9, 5, 9, src=20)
    run(10, 0, 8)
    run(11, 3, S - 3, src=21)
    run(12, S // 2, 1, src=22)
    for p in range(13, 19):
        run(p, (7 * p) % S, 1)
    x = torch.randn(len(slots), 2, heads, D, generator=g)
    x[2] = 0
    x[-3:] = 0  # zero tokens: a zero scale where the block is new
    check_append(x.to(dtype), cache, slots, sources, spread=heads > 1)
    check_append(x.to(dtype), cache, slots, None)


def test_append_values_that_are_not_numbers_or_tiny():
    g = gen(3)
    cache = new_cache(g, 4, 1, 16, 64)
    x = torch.randn(5, 2, 1, 64, generator=g)
    x[0, 0, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, -0.0])
    x[1] = math.inf
    x[2] = 2.0 ** -110
    x[3] = 3e38
    x[4] = math.nan
    check_append(x.bfloat16(), cache, [0, 16, 33, 48, 49], None)
    check_append(x[2:3].bfloat16(), cache, [32], None)
    check_append(x[4:5].bfloat16(), cache, [0], None)


def test_append_skips_slots_outside_the_cache():
    g = gen(4)
    cache = new_cache(g, 3, 2, 16, 64)
    x = torch.randn(4, 2, 2, 64, generator=g).half()
    check_append(x, cache, [48, 7, 1 << 40, 20], [0, 0, 0, 3], bad=True)


@pytest.mark.parametrize("T", [1, 5, 4000])
def test_append_long_prompt(T):
    g = gen(T)
    S, D = 32, 64
    blocks = T // S + 3
    cache = new_cache(g, blocks, 2, S, D)
    x = torch.randn(T, 2, 2, D, generator=g).bfloat16()
    slots = [7 + i for i in range(T)]
    check_append(x, cache, slots, None)


# ----------------------------------------------------------------- attend --
def make_attend(seed, lens, qs, H, G, D, S, dtype, q_scale=2.0, spare=2):
    g = gen(seed)
    R = len(lens)
    width = max(1, max(-(-max(n, 0) // S) for n in lens)) + 1
    blocks = sum(-(-max(n, 0) // S) for n in lens) + spare
    perm = torch.randperm(blocks, generator=g).tolist()
    table = []
    for n in lens:
        p = -(-max(n, 0) // S)
        table.append([perm.pop() for _ in range(p)] + [-5] * (width - p))
    codes = [torch.randint(-127, 128, (blocks, H, S, D), generator=g, dtype=torch.int8) for _ in range(2)]
    scales = [(0.2 + torch.rand(blocks, H, generator=g)) / 60 for _ in range(2)]
    start = [0]
    for m in qs:
        start.append(start[-1] + m)
    q = (q_scale * torch.randn(start[-1], H * G, D, generator=g)).to(dtype)
    return q, codes, scales, table, start, list(lens)


def check_attend(q, codes, scales, table, start, lens, scale=None, causal=True, max_q=None, max_len=None, bad=False, strided=False, empty=()):
    T, Hq, D = q.shape
    S = codes[0].shape[2]
    factor = D ** -0.5 if scale is None else scale
    seen = [0 if r in empty else n for r, n in enumerate(lens)]
    want, parts = ref.attend(q, codes[0], codes[1], scales[0], scales[1], table, start, seen, factor, causal)
    tol = ref.attend_tolerance(want, parts, q.dtype, D)
    dq = q.cuda()
    out = None
    if strided:  # a slice of a fused projection, and a wider output
        wide = torch.full((T, Hq + 3, D), 9.0, dtype=q.dtype, device="cuda")
        wide[:, 1:1 + Hq] = dq
        dq = wide[:, 1:1 + Hq]
        hold = torch.full((T, 2 * Hq, D), 7.0, dtype=q.dtype, device="cuda")
        out = hold[:, ::2]
    cache = st.KvCache(codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda())
    got = st.st_kv_attend(cache, dq, torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor(start, dtype=torch.int32).cuda(),
                          torch.tensor(lens, dtype=torch.int32).cuda(), max_q or max(1, max(b - a for a, b in zip(start, start[1:]))),
                          max_len=max_len, scale=scale, causal=causal, out=out)
    assert st.st_decode_check() == (st.ST_ERR_DEVICE if bad else st.ST_OK)
    got64 = got.cpu().double()
    n = start[-1]
    strange = ~q[:n].isfinite().all(-1, keepdim=True) & (want[:n].isnan().any(-1, keepdim=True))
    assert torch.equal(got64[:n].isnan(), strange.expand_as(got64[:n]))
    off = (got64[:n] - want[:n]).abs() - tol[:n]
    off[strange.expand_as(off)] = -1
    assert bool((off <= 0).all()), f"off by {float(off.max()):.3g} over the tolerance"
    if strided:
        assert bool((hold[:, 1::2] == 7.0).all())
    return got


LENS = [
    ([1], [1]),
    ([0, 1, 2, 17], [1, 1, 1, 1]),
    ([15, 16, 17, 33, 64, 65, 127, 128, 129], [1] * 9),
    ([700, 3, 0, 129, 1300], [1] * 5),
    ([40, 5, 200], [3, 5, 8]),
    ([70, 300, 1], [70, 33, 1]),
    ([600], [257]),
]


@pytest.mark.parametrize("lens,qs", LENS)
@pytest.mark.parametrize("H,G,D,S,dtype", [
    (1, 1, 64, 16, torch.float16), (2, 4, 128, 32, torch.bfloat16), (1, 8, 128, 64, torch.float16),
    (3, 5, 64, 128, torch.bfloat16), (1, 16, 128, 16, torch.bfloat16), (2, 3, 128, 128, torch.float16), (1, 40, 64, 64, torch.bfloat16)])
def test_attend(lens, qs, H, G, D, S, dtype):
    check_attend(*make_attend(len(lens) + G, lens, qs, H, G, D, S, dtype))


@pytest.mark.parametrize("S,D", [(16, 64), (64, 128)])
def test_attend_long_rows_are_split_and_joined(S, D):
    check_attend(*make_attend(1, [9001, 4097, 10], [1, 1, 1], 1, 4, D, S, torch.bfloat16))
    check_attend(*make_attend(2, [5000, 12], [4, 2], 2, 2, D, S, torch.float16))


def test_attend_mixed_batches():
    """Rows of single tokens beside prompts: each kind in its kernel, both of them split and joined."""
    check_attend(*make_attend(20, [3000, 40, 2500, 0, 1, 5000], [1, 40, 300, 1, 1, 9], 1, 4, 64, 16, torch.bfloat16))
    check_attend(*make_attend(21, [700, 2600, 90, 33], [2, 200, 90, 33], 2, 8, 128, 32, torch.float16))
    check_attend(*make_attend(22, [300] * 40, [1] * 20 + [17] * 20, 1, 3, 64, 64, torch.bfloat16))
    check_attend(*make_attend(23, [260, 80], [1, 80], 1, 40, 64, 16, torch.float16))  # more heads than the small kernel takes


@pytest.mark.parametrize("max_len", [None, 2510])
def test_attend_rows_with_more_queries_than_said(max_len):
    """Zeros for them, the others as ever."""
    q, codes, scales, table, start, lens = make_attend(24, [2500, 60, 100, 50], [70, 3, 40, 50], 1, 4, 64, 16, torch.float16)
    got = check_attend(q, codes, scales, table, start, lens, max_q=50, max_len=max_len, bad=True, empty=(0,))
    assert bool((got[:70] == 0).all())
    got = check_attend(q, codes, scales, table, start, lens, max_q=2, max_len=max_len, bad=True, empty=(0, 1, 2, 3))
    assert bool((got == 0).all())


def test_attend_strided_and_not_causal():
    a = make_attend(5, [100, 31], [9, 31], 2, 3, 64, 16, torch.bfloat16)
    check_attend(*a, strided=True)
    check_attend(*a, causal=False, strided=True)
    check_attend(*make_attend(6, [300], [1], 2, 2, 128, 32, torch.float16), strided=True)


def test_attend_more_queries_than_tokens_gives_zero_rows():
    q, codes, scales, table, start, lens = make_attend(7, [5, 3], [12, 3], 1, 2, 64, 16, torch.float16)
    got = check_attend(q, codes, scales, table, start, lens)
    assert bool((got[:7] == 0).all()) and bool((got[7:12] != 0).any())
    check_attend(q, codes, scales, table, start, [-1, 3])


def test_attend_large_and_tiny_queries():
    for q_scale, dtype in ((300.0, torch.bfloat16), (1e30, torch.bfloat16), (1e-30, torch.bfloat16), (20000.0, torch.float16), (1e-6, torch.float16)):
        a = make_attend(8, [130, 20], [1, 20], 1, 4, 64, 16, dtype, q_scale=q_scale)
        check_attend(*a, scale=0.125 / q_scale)
    zero = make_attend(8, [130, 20], [1, 20], 1, 4, 64, 16, torch.bfloat16, q_scale=0.0)
    check_attend(*zero)


def test_attend_queries_that_are_not_numbers():
    """NaN in the heads that hold one, nowhere else."""
    q, codes, scales, table, start, lens = make_attend(16, [130, 20, 0], [1, 20, 1], 2, 4, 64, 16, torch.bfloat16)
    q[0, 1, 5], q[7, 2, 63], q[20, 7, 0], q[21, 3, 1] = math.inf, -math.inf, math.nan, math.nan
    check_attend(q, codes, scales, table, start, lens)


def test_attend_one_weight_takes_all():
    """Scores far apart: the softmax is one key's."""
    a = make_attend(9, [257, 40], [2, 40], 1, 2, 128, 32, torch.bfloat16, q_scale=40.0)
    check_attend(*a)


@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_many_small_weights_make_up_the_sum(queries, D):
    """One key takes all of the softmax but its value is 0; each of the others weighs 2^-22 of it. Tolerance: the output's
    half step, the weights' rounding to 11 bits or 2^-32 (2^-10 of 2^-22), 2^-16 for fp32 scores near 22 and sums."""
    n, S = 40000, 64
    blocks = n // S
    codes = [torch.zeros(blocks, 1, S, D, dtype=torch.int8) for _ in range(2)]
    codes[0][3, 0, 5, 0] = 100
    codes[1][:] = 100
    codes[1][3, 0, 5] = 0
    scales = [torch.full((blocks, 1), 0.25) for _ in range(2)]
    q = torch.zeros(queries, 1, D)
    q[..., 0] = 1.0
    got = st.st_kv_attend(st.KvCache(*(x.cuda() for x in codes), *(x.cuda() for x in scales)), q.half().cuda(),
                          torch.arange(blocks, dtype=torch.int32)[None].cuda(), torch.tensor([0, queries], dtype=torch.int32).cuda(),
                          torch.tensor([n], dtype=torch.int32).cuda(), queries, scale=22 * math.log(2) / 25, causal=False)
    want = 25.0 * (n - 1) * 2.0 ** -22 / (1 + (n - 1) * 2.0 ** -22)
    assert bool(((got.cpu().double() - want).abs() <= want * (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -16)).all())


def test_attend_tiny_value_scales():
    """V scales below fp32's normal numbers, as a caller's own cache may hold."""
    q, codes, scales, table, start, lens = make_attend(14, [300, 90], [1, 40], 1, 2, 64, 16, torch.bfloat16)
    scales[1][:] = 2.0 ** -140
    got = check_attend(q, codes, scales, table, start, lens)
    assert bool(got.isfinite().all())


def test_attend_scales_of_blocks_far_apart_and_zero():
    q, codes, scales, table, start, lens = make_attend(10, [400, 90], [1, 5], 2, 4, 64, 16, torch.float16)
    for i in range(2):
        scales[i] *= torch.exp2(torch.randint(-12, 1, scales[i].shape, generator=gen(i)).float())
    scales[1][table[0][3]] = 0
    scales[1][table[1][0]] = 0
    check_attend(q, codes, scales, table, start, lens)
    scales[1][:] = 0
    assert bool((check_attend(q, codes, scales, table, start, lens) == 0).all())


def test_attend_codes_of_minus_128():
    q, codes, scales, table, start, lens = make_attend(11, [77], [3], 1, 2, 64, 16, torch.bfloat16)
    codes[0][codes[0] < -60] = -128
    codes[1][codes[1] > 60] = -128
    check_attend(q, codes, scales, table, start, lens)


@pytest.mark.parametrize("qs", [[1, 1], [40, 20]])
def test_attend_hides_bad_blocks_and_marks_the_error_word(qs):
    q, codes, scales, table, start, lens = make_attend(12, [100, 50], qs, 1, 2, 64, 16, torch.float16)
    table[0][2] = -1
    table[1][0] = 10 ** 6
    check_attend(q, codes, scales, table, start, lens, bad=True)


@pytest.mark.parametrize("qs", [[1, 1, 1], [40, 3, 20]])
def test_attend_rows_longer_than_said(qs):
    a = make_attend(13, [200, 90, 30], qs, 1, 2, 64, 16, torch.float16)
    got = check_attend(*a, max_len=100, bad=True, empty=(0,))
    assert bool((got[:qs[0]] == 0).all())


@pytest.mark.parametrize("qs", [[1, 1], [30, 20]])
def test_attend_leaves_rows_behind_the_last_sequence(qs):
    q, codes, scales, table, start, lens = make_attend(14, [100, 50], qs, 2, 2, 64, 32, torch.float16)
    n = start[-1]
    q = torch.cat([q, torch.full((5,) + q.shape[1:], math.nan, dtype=q.dtype)])
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    cache = st.KvCache(codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda())
    args = (torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor(start, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    st.st_kv_attend(cache, q.cuda(), *args, max(qs), out=out)
    assert bool((out[n:] == 3.0).all()) and bool((out[:n] != 3.0).any())


def test_attend_masked_places_may_hold_anything():
    """Scales that are NaN and infinite behind a row's last block, and in blocks of no row, are not read."""
    q, codes, scales, table, start, lens = make_attend(15, [100, 50], [1, 7], 2, 2, 64, 16, torch.bfloat16, spare=6)
    used = {p for row, n in zip(table, lens) for p in row[:-(-n // 16)]}
    for p in range(codes[0].shape[0]):
        if p not in used:
            scales[0][p], scales[1][p] = math.nan, math.inf
    check_attend(q, codes, scales, table, start, lens)


def test_attend_and_append_in_a_cache_beyond_32_bit_offsets():
    """Keys and values of 4.5 GB each, the rows' blocks at both ends."""
    S, H, D = 128, 8, 128
    blocks = (9 << 29) // (H * S * D) + 3
    cache = st.KvCache(torch.empty(blocks, H, S, D, dtype=torch.int8, device="cuda"), torch.empty(blocks, H, S, D, dtype=torch.int8, device="cuda"),
                       torch.empty(blocks, H, device="cuda"), torch.empty(blocks, H, device="cuda"))
    pages = [blocks - 1, 0, blocks - 2, 1, blocks // 2]
    n = 4 * S + 37
    g = gen(30)
    x = torch.randn(n, 2, H, D, generator=g).bfloat16()
    slots = [pages[i // S] * S + i % S for i in range(n)]
    small = [torch.zeros(5, H, S, D, dtype=torch.int8), torch.zeros(5, H, S, D, dtype=torch.int8), torch.zeros(5, H), torch.zeros(5, H)]
    for i in range(2):
        codes, scales = small[i].numpy(), small[2 + i].numpy()
        ref.append(codes, scales, x[:, i].float().numpy(), [i // S * S + i % S for i in range(n)], None)
    st.st_kv_append(cache, x[:, 0].cuda(), x[:, 1].cuda(), torch.tensor(slots).cuda())
    for i, p in enumerate(pages):
        m = min(S, n - i * S)
        assert torch.equal(cache.k[p, :, :m].cpu(), small[0][i, :, :m]) and torch.equal(cache.v[p, :, :m].cpu(), small[1][i, :, :m])
        assert torch.equal(cache.k_scale[p].cpu(), small[2][i]) and torch.equal(cache.v_scale[p].cpu(), small[3][i])
    for m in (1, 90):
        q = torch.randn(m, 2 * H, D, generator=g).bfloat16()
        want, parts = ref.attend(q, small[0], small[1], small[2], small[3], [[0, 1, 2, 3, 4]], [0, m], [n], D ** -0.5)
        got = st.st_kv_attend(cache, q.cuda(), torch.tensor([pages], dtype=torch.int32).cuda(), torch.tensor([0, m], dtype=torch.int32).cuda(),
                              torch.tensor([n], dtype=torch.int32).cuda(), m)
        assert bool(((got.cpu().double() - want).abs() <= ref.attend_tolerance(want, parts, torch.bfloat16, D)).all())
    assert st.st_decode_check() == st.ST_OK


@pytest.mark.parametrize("qs", [[1, 1], [3, 90, 1], [200]])
def test_attend_in_place(qs):
    """The output may take the queries' place."""
    q, codes, scales, table, start, lens = make_attend(41, [3000 + m for m in qs], qs, 2, 4, 64, 16, torch.bfloat16)
    cache = st.KvCache(codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda())
    q = q.cuda()
    args = [torch.tensor(x, dtype=torch.int32).cuda() for x in (table, start, lens)] + [max(qs)]
    want = st.st_kv_attend(cache, q, *args)
    got = st.st_kv_attend(cache, q, *args, out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


# ----------------------------------------------------------------- select --
def check_select(logits, scores, keep, allow=None, finished=None, end=0):
    cuda = lambda x: None if x is None else x.cuda()  # noqa: E731
    s, p, t, f = st.st_beam_select(cuda(logits), cuda(scores), keep, allow=cuda(allow), finished=cuda(finished), end_token=end)
    s, p, t = s.cpu(), p.cpu(), t.cpu()
    for b, want in enumerate(ref.select(logits, scores, keep, allow, finished, end)):
        n = len(want)
        assert p[b].tolist() == [w[1] for w in want] + [-1] * (keep - n)
        assert t[b].tolist() == [w[2] for w in want] + [-1] * (keep - n)
        assert bool((s[b, n:] == -math.inf).all())
        w = torch.tensor([x[0] for x in want], dtype=torch.float64)
        # one rounding of the 64-bit score to fp32
        assert bool(((s[b, :n].double() - w).abs() <= w.abs() * 2.0 ** -24 + 1e-11).all())
        if finished is not None:
            assert f[b].tolist() == [bool(finished[b, x[1]]) or x[2] == end for x in want] + [False] * (keep - n)
    return s, p, t


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,K,V,keep", [
    (1, 1, 1, 1), (1, 1, 5, 9), (3, 4, 7, 4), (2, 3, 300, 64), (2, 16, 1021, 16), (1, 4, 8192, 8), (2, 2, 8193, 200),
    (1, 3, 16385, 512), (1, 5, 50001, 10), (2, 256, 33, 512), (1, 64, 2000, 128), (1, 1, 100003, 300)])
def test_select(B, K, V, keep, dtype):
    g = gen(B * K + V)
    logits = (3 * torch.randn(B, K, V, generator=g)).to(dtype)
    check_select(logits, -10 * torch.rand(B, K, generator=g), keep)


@pytest.mark.parametrize("B,K,V,keep", [(2, 4, 100, 8), (3, 16, 1021, 32), (2, 3, 20001, 6)])
def test_select_masked_and_finished(B, K, V, keep):
    g = gen(V)
    logits = (3 * torch.randn(B, K, V, generator=g)).bfloat16()
    logits[..., ::7] = math.nan
    logits[..., 3::11] = math.inf
    logits[..., 5::13] = -math.inf
    scores = -10 * torch.rand(B, K, generator=g)
    words = torch.randint(-2**31, 2**31 - 1, (B, K, -(-V // 32)), generator=g).int()
    words[0, 1] = 0  # a beam that may take nothing
    finished = torch.rand(B, K, generator=g) < 0.4
    check_select(logits, scores, keep)
    check_select(logits, scores, keep, allow=words)
    check_select(logits, scores, keep, allow=words[:, :1].expand(B, K, -1))
    check_select(logits, scores, keep, allow=words[:1, :1].expand(B, K, -1), finished=finished, end=V - 1)
    scores[0, 0], scores[1, 1], scores[1, 2] = -math.inf, math.nan, math.inf
    check_select(logits, scores, keep, finished=finished, end=2)
    check_select(logits, torch.full((B, K), -math.inf), keep, allow=words)
    check_select(logits, scores, keep, finished=torch.ones(B, K, dtype=torch.bool), end=0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V,keep", [(2, 4, 1000, 16), (1, 2, 30011, 500), (1, 256, 9000, 512), (1, 200, 64, 300)])
def test_select_ties_go_to_the_lowest_index(B, K, V, keep, dtype):
    g = gen(V)
    same = torch.zeros(B, K, V, dtype=dtype)
    check_select(same, torch.zeros(B, K), keep)
    few = torch.randint(0, 3, (1, 1, V), generator=g).to(dtype).expand(B, K, V).contiguous()
    check_select(few, torch.zeros(B, K), keep)
    signed = torch.where(torch.rand(B, K, V, generator=g) < 0.5, 0.0, -0.0).to(dtype)
    check_select(signed, torch.zeros(B, K), keep)


def test_select_first_step_has_one_living_beam():
    g = gen(2)
    logits = torch.randn(4, 6, 500, generator=g)
    scores = torch.full((4, 6), -math.inf)
    scores[:, 0] = 0
    _, parents, _ = check_select(logits, scores, 6)
    assert bool((parents == 0).all())


def test_select_strided_and_unaligned_rows():
    g = gen(9)
    for dtype in (torch.bfloat16, torch.float32):
        for pad, shift in ((0, 1), (3, 0), (5, 3)):
            base = (3 * torch.randn(2 * 5 * (801 + pad) + shift, generator=g)).to(dtype)
            x = base[shift:].view(2, 5, 801 + pad)[..., :801]
            s = -torch.rand(2, 5, generator=g)
            d = base.cuda()[shift:].view(2, 5, 801 + pad)[..., :801]
            got = st.st_beam_select(d, s.cuda(), 20)
            want = st.st_beam_select(x.contiguous().cuda(), s.cuda(), 20)
            assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
            check_select(x.contiguous(), s, 20)


def test_select_logits_beyond_32_bit_offsets():
    g = gen(31)
    step = (1 << 30) + 12
    base = torch.zeros(2 * step + 1000, dtype=torch.bfloat16, device="cuda")
    x = (3 * torch.randn(1, 3, 1000, generator=g)).bfloat16()
    d = base.as_strided((1, 3, 1000), (3 * step, step, 1))
    d.copy_(x)
    s = -torch.rand(1, 3, generator=g)
    got = st.st_beam_select(d, s.cuda(), 30)
    want = st.st_beam_select(x.cuda(), s.cuda(), 30)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    check_select(x, s, 30)


def test_select_far_apart_logits():
    """Ranges that overflow fp32, and values next to each other in fp32."""
    x = torch.zeros(1, 3, 40)
    x[0, 0, ::3] = 3e38
    x[0, 0, 1::3] = -3e38
    x[0, 1] = 100 + torch.arange(40) * 2.0 ** -17
    x[0, 2, 5] = -3.3e38
    check_select(x, torch.tensor([[0.0, -1e-3, -2.0]]), 60)
    check_select(x, torch.tensor([[-3e38, -1e-3, 3e38]]), 60)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K,V,pad,shift", [(7, 3001, 0, 0), (9, 70003, 0, 1), (5, 20000, 3, 2), (256, 33, 0, 0)])
def test_select_equal_beams_stand_in_order(K, V, pad, shift, dtype):
    """Beams with the same logits and scores have the same normaliser to the last bit, however their rows are aligned."""
    g = gen(V + K)
    row = (3 * torch.randn(V, generator=g)).to(dtype)
    base = torch.zeros(K * (V + pad) + shift, dtype=dtype)
    x = base[shift:].view(1, K, V + pad)[..., :V]
    x.copy_(row.expand(1, K, V))
    keep = min(512, 3 * K)
    want = torch.sort(row.float().repeat(K), descending=True, stable=True).indices[:keep]
    scores, parents, tokens, _ = st.st_beam_select(base.cuda()[shift:].view(1, K, V + pad)[..., :V], torch.full((1, K), -2.5).cuda(), keep)
    assert parents[0].tolist() == (want // V).tolist() and tokens[0].tolist() == (want % V).tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("centre", [300.0, -16000.0, 16600.0, 60000.0])
def test_select_logits_far_from_zero(centre, dtype):
    x = (torch.linspace(-9, 3, 2 * 3 * 9001)[torch.randperm(2 * 3 * 9001, generator=gen(int(abs(centre))))].view(2, 3, 9001) + centre).to(dtype)
    check_select(x, -torch.rand(2, 3, generator=gen(3)), 40)


def test_select_many_rows_go_in_several_launches():
    g = gen(1)
    logits = torch.randn(4400, 16, 8, generator=g)
    scores = -torch.rand(4400, 16, generator=g)
    words = torch.randint(0, 256, (4400, 16, 1), generator=g).int()
    check_select(logits, scores, 16, allow=words)


# ---------------------------------------------------------------- reorder --
@pytest.mark.parametrize("shape,dtype", [((3, 4, 7), torch.int32), ((2, 5, 3, 16), torch.bfloat16), ((1, 1, 1), torch.int8), ((4, 3, 70001), torch.int8),
                                         ((2, 8, 40000), torch.float32), ((5, 2, 33), torch.float16), ((2, 3), torch.float32), ((70, 1, 5), torch.bool)])
@pytest.mark.parametrize("keep", [1, 3, 8])
def test_reorder(shape, dtype, keep):
    g = gen(sum(shape))
    B, K = shape[:2]
    x = torch.randint(0, 2 if dtype == torch.bool else 100, shape, generator=g).to(dtype).cuda()
    y = torch.randn((B, K, 13), generator=g).cuda()
    parents = torch.randint(-1, K, (B, keep), generator=g).int()
    got = st.st_beam_reorder([x, y], parents.cuda())
    assert st.st_decode_check() == st.ST_OK
    for src, dst in ((x, got[0]), (y, got[1])):
        for b in range(B):
            for j in range(keep):
                p = int(parents[b, j])
                want = torch.zeros_like(src[b, 0]) if p < 0 else src[b, p]
                assert torch.equal(dst[b, j], want)


def test_reorder_layers_strides_and_out():
    g = gen(4)
    big = torch.randn(5, 3, 4, 2, 24, generator=g).cuda()
    x = big[:, :, :, 1]  # rows with a gap between them
    parents = torch.randint(0, 4, (3, 6), generator=g).int().cuda()
    hold = torch.full((5, 3, 6, 30), 2.0, device="cuda")
    out = hold[..., :24]
    got = st.st_beam_reorder([x], parents, out=[out], beam_dim=2)[0]
    want = torch.stack([torch.stack([x[:, b, parents[b].long()] for b in range(3)], 1)])[0]
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
    assert bool((hold[..., 24:] == 2.0).all())


def test_reorder_beyond_32_bit_offsets():
    n = (5 << 28) + 16
    x = torch.zeros(1, 4, n, dtype=torch.int8, device="cuda")
    for i in range(4):
        x[0, i, 0], x[0, i, -1] = 10 + i, 20 + i
    got = st.st_beam_reorder([x], torch.tensor([[3, 0, -1, 2]], dtype=torch.int32).cuda())[0]
    assert got[0, :, 0].tolist() == [13, 10, 0, 12] and got[0, :, -1].tolist() == [23, 20, 0, 22] and int(got.sum()) == 100


def test_reorder_bad_parents_give_zeros_and_the_error_word():
    x = torch.ones(2, 3, 20, device="cuda")
    got = st.st_beam_reorder([x], torch.tensor([[0, 3], [-2, 1]], dtype=torch.int32).cuda())[0]
    assert st.st_decode_check() == st.ST_ERR_DEVICE
    assert got.sum(-1).tolist() == [[20, 0], [0, 20]]
    assert st.st_decode_check() == st.ST_OK


def test_reorder_refuses_overlap():
    x = torch.zeros(2, 3, 8, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for out in (x, x.view(-1)[:].view(2, 3, 8)):
        with pytest.raises(st.StError) as e:
            st.st_beam_reorder([x], p, out=[out])
        assert e.value.status == st.ST_ERR_INVALID_ARG
    y = torch.zeros(2, 3, 8, device="cuda")
    with pytest.raises(st.StError):
        st.st_beam_reorder([x, x], p, out=[y, y])
    with pytest.raises(st.StError):
        st.st_beam_reorder([x], p, out=[torch.zeros(1, 1, 8, device="cuda").expand(2, 3, 8)])
