"""What the decode calls refuse, without a GPU: bad sizes in the C calls, bad
tensors in the binding. None of these gets as far as a launch."""
import ctypes

import pytest
import torch

import filtered_int8_ann_b200 as st
from filtered_int8_ann_b200 import build

P = ctypes.c_void_p
FAKE = P(4096)
BAD, UNSUPPORTED = st.ST_ERR_INVALID_ARG, st.ST_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return st.lib()


def cache(blocks=8, heads=2, size=16, dim=64):
    c = st._KvCache(4096, 4096, 4096, 4096, blocks, heads, size, dim)
    return ctypes.byref(c)


def plan(lib, R=2, width=4, blocks=8, size=16, T=3, **k):
    p = lambda n: k.get(n, FAKE)  # noqa: E731
    return lib.st_kv_plan(p("table"), p("have"), p("add"), R, width, blocks, size, T, p("slots"), p("sources"), FAKE, FAKE, FAKE, None)


def test_plan_sizes(lib):
    assert plan(lib, R=0) == BAD and plan(lib, width=0) == BAD and plan(lib, blocks=0) == BAD
    assert plan(lib, T=-1) == BAD and plan(lib, size=24) == BAD and plan(lib, size=0) == BAD and plan(lib, size=256) == BAD
    assert plan(lib, R=32769) == UNSUPPORTED and plan(lib, blocks=4194305) == UNSUPPORTED
    assert plan(lib, T=2**31) == UNSUPPORTED and plan(lib, R=32768, width=65536) == UNSUPPORTED


def append(lib, c, dtype=0, T=3, kt=128, kh=64, vt=128, vh=64):
    return lib.st_kv_append(c, FAKE, FAKE, dtype, T, kt, kh, vt, vh, FAKE, FAKE, None)


def test_cache_sizes(lib):
    for c in (cache(blocks=0), cache(heads=0), cache(size=0), cache(dim=0), None):
        assert append(lib, c) == BAD
    for c in (cache(blocks=4194305), cache(heads=1025), cache(size=48), cache(dim=96), cache(dim=256)):
        assert append(lib, c) == UNSUPPORTED
    assert append(lib, cache(), T=0) == st.ST_OK
    assert append(lib, cache(), T=-1) == BAD and append(lib, cache(), T=2**31) == UNSUPPORTED
    assert append(lib, cache(), dtype=2) == BAD and append(lib, cache(), dtype=7) == BAD
    assert append(lib, cache(), kt=4) == BAD and append(lib, cache(), vh=-8) == BAD


def attend(lib, c, dtype=0, T=3, heads=4, qt=256, qh=64, width=4, R=2, max_q=1, max_len=64, scale=1.0, ot=256, oh=64):
    return lib.st_kv_attend(c, FAKE, dtype, T, heads, qt, qh, FAKE, width, FAKE, FAKE, R, max_q, max_len, scale, 1, FAKE, ot, oh, None, 0, None)


def test_attend_sizes(lib):
    c = cache()
    for k in (dict(heads=3), dict(heads=0), dict(R=0), dict(max_q=0), dict(max_q=2**20 + 1), dict(max_len=0), dict(max_len=65), dict(T=-1),
              dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=2), dict(qt=4), dict(qh=-8), dict(ot=12), dict(width=0)):
        assert attend(lib, c, **k) == BAD, k
    assert attend(lib, c, R=32769) == UNSUPPORTED and attend(lib, c, T=2**31) == UNSUPPORTED
    assert attend(lib, cache(dim=96)) == UNSUPPORTED and attend(lib, None) == BAD
    assert attend(lib, c, T=0) == st.ST_OK
    need = ctypes.c_int64(-1)
    assert lib.st_kv_attend_workspace(c, 3, 4, 2, 1, 64, ctypes.byref(need)) == st.ST_OK and need.value >= 0
    assert lib.st_kv_attend_workspace(c, 3, 4, 0, 1, 64, ctypes.byref(need)) == BAD and need.value == 0
    assert lib.st_kv_attend_workspace(c, 3, 4, 2, 1, 64, None) == BAD


def select(lib, dtype=0, stride=100, B=2, K=3, V=100, keep=4, ex=None):
    return lib.st_beam_select(FAKE, dtype, stride, FAKE, B, K, V, keep, FAKE, FAKE, FAKE, ex, None, 0, None)


def test_select_sizes(lib):
    for k in (dict(B=0), dict(K=0), dict(V=0), dict(keep=0), dict(stride=99), dict(dtype=3), dict(dtype=-1)):
        assert select(lib, **k) == BAD, k
    for k in (dict(B=32769), dict(K=257), dict(keep=513), dict(V=2**20 + 1, stride=2**21)):
        assert select(lib, **k) == UNSUPPORTED, k
    one = st._BeamExtras(finished=4096)
    assert select(lib, ex=ctypes.byref(one)) == BAD
    end = st._BeamExtras(finished=4096, out_finished=4096, end_token=100)
    assert select(lib, ex=ctypes.byref(end)) == BAD
    back = st._BeamExtras(allow=4096, allow_beam_stride=-1)
    assert select(lib, ex=ctypes.byref(back)) == BAD
    need = ctypes.c_int64(-1)
    assert lib.st_beam_select_workspace(2, 3, 100, 4, ctypes.byref(need)) == st.ST_OK
    assert lib.st_beam_select_workspace(2, 300, 100, 4, ctypes.byref(need)) == UNSUPPORTED and need.value == 0


def test_reorder_sizes(lib):
    s = (st._BeamState * 17)()
    call = lambda n=1, B=1, K=1, keep=1, p=FAKE: lib.st_beam_reorder(s, n, p, B, K, keep, None)  # noqa: E731
    assert lib.st_beam_reorder(None, 1, FAKE, 1, 1, 1, None) == BAD
    assert call(n=0) == BAD and call(B=0) == BAD and call(K=0) == BAD and call(keep=0) == BAD
    assert call(n=17) == UNSUPPORTED and call(B=2**20, K=2**11) == UNSUPPORTED
    s[0].row_bytes = -1
    assert call() == BAD


def test_binding_refuses_wrong_tensors():
    z = torch.zeros
    i32 = torch.int32
    k, sc = z(4, 2, 16, 64, dtype=torch.int8), z(4, 2)
    for bad in ((k.short(), k, sc, sc), (k, k[:3], sc, sc), (k, k, sc.double(), sc), (k, k, sc, sc[:, :1]), (k[:, :, :, ::2], k, sc, sc), (k[0], k, sc, sc)):
        with pytest.raises(ValueError):
            st.KvCache(*bad)
    c = st.KvCache(k, k.clone(), sc, sc.clone())
    x = z(3, 2, 64, dtype=torch.bfloat16)
    slots = z(3, dtype=torch.int64)
    for a in ((x.float(), x, slots), (x, x.half(), slots), (x[:, :1], x, slots), (x, x[:2], slots), (x, x, slots.int()), (x[..., :32], x, slots),
              (z(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2), x, slots), (x, x, slots, slots)):
        with pytest.raises(ValueError):
            st.st_kv_append(c, *a)
    table, start, lens = z(2, 4, dtype=i32), z(3, dtype=i32), z(2, dtype=i32)
    for a in ((x.float(), table, start, lens), (x, table.long(), start, lens), (x, table, start[:2], lens), (x, table, start, lens.float()), (x, table[0], start, lens)):
        with pytest.raises(ValueError):
            st.st_kv_attend(c, *a, 1)
    with pytest.raises(ValueError):
        st.st_kv_attend(c, x, table, start, lens, 1, out=x[:, :1].expand(3, 2, 64))
    with pytest.raises(ValueError):
        st.st_kv_plan(table, lens, start, 8, 16, 3)
    with pytest.raises(ValueError):
        st.st_kv_plan(table.t(), z(4, dtype=i32), z(4, dtype=i32), 8, 16, 3)
    logits, scores = z(2, 3, 50), z(2, 3)
    for a, kw in (((logits.double(), scores, 4), {}), ((logits[0], scores, 4), {}), ((logits, scores[:1], 4), {}), ((logits[..., ::2], scores, 4), {}),
                  ((logits, scores, 4), dict(allow=z(2, 3, 1, dtype=i32))), ((logits, scores, 4), dict(finished=z(2, 3))), ((z(4, 3, 50)[::2], scores, 4), {})):
        with pytest.raises(ValueError):
            st.st_beam_select(*a, **kw)
    parents = z(2, 3, dtype=i32)
    for a, kw in ((([], parents), {}), (([z(2, 3, 4), z(2, 4, 4)], parents), {}), (([z(3, 3, 4)], parents), {}), (([z(2, 3, 4)], parents[0]), {}),
                  (([z(2, 3, 4, 4).transpose(2, 3)], parents), {}), (([z(2, 3, 4)], parents), dict(out=[z(2, 4, 4)])), (([z(2, 3, 4)], parents.long()), {}),
                  (([z(4, 3, 4)[::2]], parents), {})):
        with pytest.raises(ValueError):
            st.st_beam_reorder(*a, **kw)


def test_binding_refuses_host_tensors():
    """Well-formed tensors of the host."""
    z = torch.zeros
    i32 = torch.int32
    logits, scores = z(2, 3, 50), z(2, 3)
    with pytest.raises(ValueError, match="CUDA device"):
        st.st_beam_select(logits, scores, 4)
    with pytest.raises(ValueError, match="CUDA device"):
        st.st_beam_reorder([logits], z(2, 3, dtype=i32))
    with pytest.raises(ValueError, match="CUDA device"):
        st.st_kv_plan(z(2, 4, dtype=i32), z(2, dtype=i32), z(2, dtype=i32), 8, 16, 3)
    k, sc = z(4, 2, 16, 64, dtype=torch.int8), z(4, 2)
    c = st.KvCache(k, k.clone(), sc, sc.clone())
    x = z(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        st.st_kv_attend(c, x, z(2, 4, dtype=i32), z(3, dtype=i32), z(2, dtype=i32), 1)
    # with every array given, the library refuses them (or, without a GPU, CUDA does)
    with pytest.raises(st.StError):
        st.st_beam_reorder([logits], z(2, 3, dtype=i32), out=[z(2, 3, 50)])
    with pytest.raises(st.StError):
        st.st_kv_append(c, x, x, z(3, dtype=torch.int64))


def test_cache_fields_do_not_change():
    c = st.KvCache.empty(4, 1, 16, 64, device="cpu")
    assert (c.num_blocks, c.kv_heads, c.block_size, c.head_dim) == (4, 1, 16, 64) and c.k.shape == c.v.shape == (4, 1, 16, 64)
    for name in ("k", "v_scale", "num_blocks"):
        with pytest.raises(AttributeError):
            setattr(c, name, None)
