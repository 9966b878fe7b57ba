"""What the binding may not pass on: workspaces smaller than they look, numbers beyond 32 bits, views that conjugate or negate."""
import pytest
import torch

import filtered_int8_ann_b200 as st

I32 = torch.int32


def cache():
    k, sc = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2)
    return st.KvCache(k, k.clone(), sc, sc.clone())


def attend(max_q=1, **k):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    return st.st_kv_attend(cache(), x, torch.zeros(2, 4, dtype=I32), torch.zeros(3, dtype=I32), torch.zeros(2, dtype=I32), max_q, out=x.clone(), **k)


@pytest.mark.parametrize("room", [torch.empty(1, dtype=torch.uint8).expand(1 << 40), torch.empty(1 << 16, dtype=torch.uint8)[::2],
                                  torch.empty(1, 64, dtype=torch.uint8).expand(1 << 20, 64), 77])
def test_workspaces_that_are_not_dense(room):
    """Their elements times their size is not the memory behind their address."""
    with pytest.raises(ValueError, match="workspace"):
        attend(workspace=room)
    with pytest.raises(ValueError, match="workspace"):
        st.st_beam_select(torch.zeros(2, 3, 50), torch.zeros(2, 3), 4, workspace=room)


def test_numbers_beyond_32_bits():
    """They would be cut to their low bits, which may be in range."""
    far = 1 << 32
    table, rows = torch.zeros(2, 4, dtype=I32), torch.zeros(2, dtype=I32)
    given = dict(slots=torch.zeros(3, dtype=torch.int64), sources=torch.zeros(3, dtype=I32), row_start=torch.zeros(3, dtype=I32), lens=rows.clone(), report=torch.zeros(4, dtype=I32))
    logits, scores = torch.zeros(2, 3, 50), torch.zeros(2, 3)
    meta = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="meta")  # noqa: E731
    for call in (lambda: st.st_kv_plan(table, rows, rows, far + 8, 16, 3, **given), lambda: st.st_kv_plan(table, rows, rows, 8, far + 16, 3, **given),
                 lambda: st.st_kv_plan(table, rows, rows, 8 - far, 16, 3, **given),
                 lambda: attend(max_q=far + 1), lambda: attend(max_q=1 - far), lambda: attend(max_len=(1 << 64) + 64),
                 lambda: st.st_beam_select(logits, scores, far + 4), lambda: st.st_beam_select(logits, scores, 4 - far),
                 lambda: st.st_beam_select(logits, scores, 4, finished=torch.zeros(2, 3, dtype=torch.bool), end_token=far),
                 lambda: st.st_beam_select(meta(1, 1, far + 50), torch.zeros(1, 1), 4),
                 lambda: st.st_beam_reorder([meta(2, far + 3, 4)], torch.zeros(2, 3, dtype=I32), out=[meta(2, 3, 4)])):
        with pytest.raises(ValueError, match="(32|64) bits"):
            call()


def test_states_that_are_conjugated_or_negated_lazily():
    """Their memory does not hold their values."""
    z = torch.complex(torch.ones(2, 3, 4), torch.ones(2, 3, 4))
    parents = torch.zeros(2, 3, dtype=I32)
    for x in (z.conj(), z.conj().imag, torch._neg_view(torch.ones(2, 3, 4))):
        for out in (None, [torch.zeros(2, 3, 4, dtype=x.dtype)]):
            with pytest.raises(ValueError, match="resolve"):
                st.st_beam_reorder([x], parents, out=out)
    with pytest.raises(ValueError, match="resolve"):
        st.st_beam_reorder([z], parents, out=[torch.zeros_like(z).conj()])
    for x, call in ((torch.zeros(3, 2, 64).bfloat16(), lambda y: st.st_kv_append(cache(), y, y, torch.zeros(3, dtype=torch.int64))),
                    (torch.zeros(2, 3, 50), lambda y: st.st_beam_select(y, torch.zeros(2, 3), 4)),
                    (torch.zeros(2, 3), lambda y: st.st_beam_select(torch.zeros(2, 3, 50), y, 4)), (torch.zeros(4, 2), lambda y: st.KvCache(cache().k, cache().v, y, y))):
        with pytest.raises(ValueError, match="resolve"):
            call(torch._neg_view(x))
