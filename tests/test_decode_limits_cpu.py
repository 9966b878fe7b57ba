"""What the decode calls ask for and refuse, without a GPU: workspaces, and arrays that may not share memory."""
import ctypes

import pytest

import filtered_int8_ann_b200 as st
from filtered_int8_ann_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return st.lib()


def attend_bytes(lib, T, R, max_q, max_len, heads=8, group=4, dim=128):
    need = ctypes.c_int64(-1)
    c = st._KvCache(None, None, None, None, 1, heads, 16, dim)
    return lib.st_kv_attend_workspace(ctypes.byref(c), T, heads * group, R, max_q, max_len, ctypes.byref(need)), need.value


@pytest.mark.parametrize("T,R,max_q,max_len,group", [
    (2517, 4, 2048, 8192, 4), (8192 + 63, 64, 8192, 65536, 4), (8192 + 63, 64, 8192, 131072, 8), (8200, 16, 2048, 131072, 4),
    (8192 + 999, 1000, 8192, 65536, 4), (70000, 3, 35000, 200000, 1)])
def test_attend_workspace_of_mixed_batches(lib, T, R, max_q, max_len, group):
    """Beside prompts, rows of up to 32 columns (query tokens x heads per cache head) need parts for those columns alone,
    however many tokens the prompts have: 128 MiB of them, or one for each 2048 cached tokens."""
    heads, part = 8, 4 * (128 + 2)
    status, need = attend_bytes(lib, T, R, max_q, max_len, group=group)
    assert status == st.ST_OK
    status, prompts = attend_bytes(lib, T, 1, max_q, max_len, group=group)  # (one row of so many columns is a prompt)
    assert status == st.ST_OK
    assert need - prompts <= max(128 << 20, R * heads * 32 * -(-max_len // 2048) * part)


def test_attend_workspace_of_single_tokens(lib):
    """Tokens behind the last row's take no part."""
    assert attend_bytes(lib, 64, 64, 1, 16384) == attend_bytes(lib, 5000, 64, 1, 16384)


@pytest.mark.parametrize("T,R,max_q,max_len,heads,group", [
    (2**31 - 1, 1, 2**20, 2**31 - 1, 1, 65535), (2**31 - 1, 7, 2**20, 2**31 - 1, 1000, 65), (2**31 - 1, 32768, 33, 2**31 - 1, 1024, 1),
    (2**31 - 1, 32768, 2**20, 2**27, 15, 4369), (2**30, 1, 2**20, 2**30, 4, 16380)])
def test_attend_workspace_that_no_memory_holds(lib, T, R, max_q, max_len, heads, group):
    """Sizes whose workspace would be more than 2^48 bytes (and more than 64 bits count) are refused."""
    assert T * heads * group * -(-max_len // 16384) * 4 * 130 > 2**48
    assert attend_bytes(lib, T, R, max_q, max_len, heads, group) == (st.ST_ERR_UNSUPPORTED, 0)


MEG = 1 << 20
BAD = st.ST_ERR_INVALID_ARG


def through(status):
    """Nothing was refused before the pointers were looked up: there is no GPU here, or the addresses are not its memory."""
    import torch
    return status == (BAD if torch.cuda.is_available() else st.ST_ERR_CUDA)


def attend_at(lib, T=6, heads=4, R=2, width=4, blocks=8, kv_heads=2, S=16, D=64, max_len=64, strides=(256, 64), out_strides=(256, 64), room=1 << 20, **at):
    """A call with every array in a megabyte of its own, but for those in `at`."""
    names = ("k", "v", "k_scale", "v_scale", "q", "out", "table", "start", "lens", "work")
    p = {n: (i + 16) * 64 * MEG for i, n in enumerate(names)}
    p.update(at)
    c = st._KvCache(p["k"], p["v"], p["k_scale"], p["v_scale"], blocks, kv_heads, S, D)
    return lib.st_kv_attend(ctypes.byref(c), p["q"], 0, T, heads, *strides, p["table"], width, p["start"], p["lens"], R, 3, max_len, 1.0, 1, p["out"], *out_strides, p["work"], room, None)


def test_attend_arrays_that_share_memory(lib):
    base = 16 * 64 * MEG
    q, out = base + 4 * 64 * MEG, base + 5 * 64 * MEG
    assert through(attend_at(lib)) and through(attend_at(lib, out=q))
    assert through(attend_at(lib, out=q + 6 * 512)) and attend_at(lib, out=q + 6 * 512 - 16) == BAD
    assert attend_at(lib, out=q + 512) == BAD and attend_at(lib, out=q, out_strides=(512, 64)) == BAD
    sizes = dict(k=8 * 2 * 16 * 64, v=8 * 2 * 16 * 64, k_scale=64, v_scale=64, table=32, start=12, lens=8)
    for n, size in sizes.items():
        assert attend_at(lib, **{n: out}) == BAD, n
        assert attend_at(lib, **{n: out + 6 * 512 - 16}) == BAD, n
        assert through(attend_at(lib, **{n: out + 6 * 512})) and through(attend_at(lib, **{n: out - size // 16 * 16 - 16})), n
    # the vectors of out among themselves
    for bad in ((0, 64), (256, 0), (256, 56), (192, 64), (64, 256)):
        assert attend_at(lib, out_strides=bad) == BAD, bad
    assert through(attend_at(lib, out_strides=(64, 6 * 64))) and through(attend_at(lib, T=1, out_strides=(0, 64)))
    # slices of one array: heads beside heads, every other head, every other token, heads outside
    assert through(attend_at(lib, strides=(1024, 64), out_strides=(1024, 64), out=q + 512))
    assert attend_at(lib, strides=(1024, 64), out_strides=(1024, 64), out=q + 496) == BAD
    assert through(attend_at(lib, strides=(512, 128), out_strides=(512, 128), out=q + 128))
    assert attend_at(lib, strides=(512, 128), out_strides=(512, 128), out=q + 64) == BAD
    assert through(attend_at(lib, strides=(512, 64), out_strides=(512, 64), out=q - 512))
    assert through(attend_at(lib, strides=(64, 1024), out_strides=(64, 1024), out=q + 6 * 128))
    assert attend_at(lib, strides=(64, 1024), out_strides=(64, 1024), out=q + 5 * 128) == BAD


def test_attend_workspace_that_shares_memory(lib):
    base = 16 * 64 * MEG
    long = dict(width=400, max_len=6400, room=8 * MEG)
    status, need = attend_bytes(lib, 6, 2, 3, 6400, 2, 2, 64)
    assert status == st.ST_OK and need > 0
    assert through(attend_at(lib, **long))
    for i, n in enumerate(("k", "v", "k_scale", "v_scale", "q", "out", "table", "start", "lens")):
        assert attend_at(lib, **long, work=base + i * 64 * MEG) == BAD, n
        assert attend_at(lib, **long, work=base + i * 64 * MEG - need + 16) == BAD, n
        assert through(attend_at(lib, **long, work=base + i * 64 * MEG - need)), n
    assert through(attend_at(lib, work=base))  # none is used


def test_attend_outputs_that_pass_share_no_byte(lib):
    """Random strides and places near the queries: what is let through is the queries' place or disjoint from them."""
    import random
    r = random.Random(1)
    q, passed = (16 + 4) * 64 * MEG, 0
    if not through(attend_at(lib)) or through(BAD):
        pytest.skip("refusals by the pointers' memory look like those for overlap")
    for _ in range(4000):
        T, heads = r.randint(1, 4), 2 * r.randint(1, 2)
        pick = lambda: r.choice([(64 * heads, 64), (64, 64 * T), (r.choice([128, 256, 512, 640]), r.choice([0, 64, 72, 128, 256]))])  # noqa: E731
        a = pick()
        b = r.choice([a, a, pick()])
        at = q + 16 * r.randint(-80, 80)
        places = lambda base, s: [base + 2 * (t * s[0] + h * s[1]) for t in range(T) for h in range(heads)]  # noqa: E731
        own, other = places(q, a), places(at, b)
        if through(attend_at(lib, T=T, heads=heads, strides=a, out_strides=b, out=at)):
            passed += 1
            assert all(abs(x - y) >= 128 for i, x in enumerate(other) for y in other[:i]), (T, heads, b)
            assert own == other or all(abs(x - y) >= 128 for x in own for y in other), (T, heads, a, b, at - q)
    assert passed > 500


def append_at(lib, T=6, blocks=8, heads=2, S=16, D=64, strides=(128, 64), **at):
    p = {n: (i + 16) * 64 * MEG for i, n in enumerate(("k", "v", "k_scale", "v_scale", "new_k", "new_v", "slots", "sources"))}
    p.update(at)
    c = st._KvCache(p["k"], p["v"], p["k_scale"], p["v_scale"], blocks, heads, S, D)
    return lib.st_kv_append(ctypes.byref(c), p["new_k"], p["new_v"], 0, T, *strides, *strides, p["slots"], p["sources"], None)


def test_append_arrays_that_share_memory(lib):
    assert through(append_at(lib)) and through(append_at(lib, sources=None))
    codes = 8 * 2 * 16 * 64
    sizes = dict(k=codes, v=codes, k_scale=64, v_scale=64, new_k=6 * 256, new_v=6 * 256, slots=48, sources=24)
    base = {n: (i + 16) * 64 * MEG for i, n in enumerate(sizes)}
    for a in ("k", "v", "k_scale", "v_scale"):
        for b in sizes:
            if a != b:
                assert append_at(lib, **{a: base[b]}) == BAD, (a, b)
                assert append_at(lib, **{a: base[b] + sizes[b] // 16 * 16 - 8}) == BAD, (a, b)
                assert through(append_at(lib, **{a: base[b] + sizes[b] + 8})) and through(append_at(lib, **{a: base[b] - sizes[a]})), (a, b)
    assert through(append_at(lib, new_v=base["new_k"])) and through(append_at(lib, strides=(0, 0)))  # both are only read
    assert append_at(lib, strides=(2**40, 64), k=base["new_k"] + 2**41) == BAD


def select_at(lib, B=2, K=3, V=100, keep=4, stride=100, allow_strides=(12, 4), extras=True, **at):
    names = ("logits", "scores", "out_scores", "out_parents", "out_tokens", "work", "allow", "finished", "out_finished")
    p = {n: (i + 16) * 64 * MEG for i, n in enumerate(names)}
    p.update(at)
    ex = st._BeamExtras(p["allow"], *allow_strides, p["finished"], p["out_finished"], 0)
    return lib.st_beam_select(p["logits"], 2, stride, p["scores"], B, K, V, keep, p["out_scores"], p["out_parents"], p["out_tokens"],
                              ctypes.byref(ex) if extras else None, p["work"], 1 << 20, None)


def test_select_arrays_that_share_memory(lib):
    need = ctypes.c_int64(0)
    assert lib.st_beam_select_workspace(2, 3, 100, 4, ctypes.byref(need)) == st.ST_OK
    sizes = dict(logits=2400, scores=24, out_scores=32, out_parents=32, out_tokens=32, work=need.value, allow=96, finished=6, out_finished=8)
    base = {n: (i + 16) * 64 * MEG for i, n in enumerate(sizes)}
    assert need.value > 0 and through(select_at(lib)) and through(select_at(lib, extras=False))
    for a in ("out_scores", "out_parents", "out_tokens", "work", "out_finished"):
        for b in sizes:
            if a != b:
                assert select_at(lib, **{a: base[b]}) == BAD, (a, b)
                assert select_at(lib, **{a: base[b] - sizes[a] + 1}) == BAD, (a, b)
                assert through(select_at(lib, **{a: base[b] + sizes[b]})) and through(select_at(lib, **{a: base[b] - sizes[a]})), (a, b)
    assert through(select_at(lib, logits=base["allow"], scores=base["finished"])) and through(select_at(lib, allow_strides=(0, 0)))  # only read
    assert through(select_at(lib, extras=False, out_scores=base["allow"], out_tokens=base["finished"]))
    assert select_at(lib, stride=2**57) == BAD and select_at(lib, allow_strides=(2**57, 4)) == BAD


def test_select_scores_may_stand_behind_the_logits(lib):
    """Outputs in the room between the beams' logits."""
    base = 16 * 64 * MEG
    assert through(select_at(lib, stride=300, out_scores=base + 400, K=1, B=1)) and select_at(lib, stride=300, out_scores=base + 396, K=1, B=1) == BAD


def test_reorder_arrays_that_share_memory(lib):
    base = 16 * MEG

    def call(parents=base, src=2 * base, dst=3 * base, src2=4 * base, dst2=5 * base, bytes2=40):
        s = (st._BeamState * 2)(st._BeamState(src, dst, 16, 16, 20, 2, 200, 300), st._BeamState(src2, dst2, bytes2, 40, 40, 1, 0, 0))
        return lib.st_beam_reorder(s, 2, parents, 2, 3, 4, None)

    assert through(call()) and through(call(src2=2 * base)) and through(call(src=base))  # only read
    span, parents = 300 + 7 * 20 + 16, 2 * 4 * 4
    for a in ("dst", "dst2"):
        size = span if a == "dst" else 8 * 40
        assert call(**{a: base}) == BAD and call(**{a: base + parents - 1}) == BAD and call(**{a: base - size + 1}) == BAD
        assert through(call(**{a: base + parents})) and through(call(**{a: base - size}))
    assert through(call(dst2=base, bytes2=0))  # skipped
    assert call(dst=2 * base) == BAD and call(dst=4 * base) == BAD and call(dst2=3 * base) == BAD


@pytest.mark.parametrize("scale,fine", [(2.35e38, True), (-2.35e38, True), (2.37e38, False), (-3.4e38, False), (float("inf"), False), (float("nan"), False)])
def test_attend_scale_in_powers_of_two(lib, scale, fine):
    """The scale times log2 e has to be an fp32 number too."""
    base = 16 * 64 * MEG
    c = st._KvCache(base, 2 * base, 3 * base, 4 * base, 8, 2, 16, 64)
    status = lib.st_kv_attend(ctypes.byref(c), 5 * base, 0, 1, 2, 0, 64, 6 * base, 4, 7 * base, 8 * base, 1, 1, 64, scale, 1, 9 * base, 0, 64, None, 0, None)
    assert through(status) if fine else status == BAD
