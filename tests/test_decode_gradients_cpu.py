"""The decode calls have no backward pass: tensors that require a gradient are refused where one would be recorded."""
import pytest
import torch

import filtered_int8_ann_b200 as st

I32 = torch.int32


def calls():
    k, sc = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2)
    cache = st.KvCache(k, k.clone(), sc, sc.clone())
    table, start, lens = torch.zeros(2, 4, dtype=I32), torch.zeros(3, dtype=I32), torch.zeros(2, dtype=I32)
    new = lambda: torch.zeros(3, 2, 64, dtype=torch.bfloat16)  # noqa: E731
    slots, parents = torch.zeros(3, dtype=torch.int64), torch.zeros(2, 3, dtype=I32)
    return {
        "k": (new(), lambda x: st.st_kv_append(cache, x, new(), slots)), "v": (new(), lambda x: st.st_kv_append(cache, new(), x, slots)),
        "q": (new(), lambda x: st.st_kv_attend(cache, x, table, start, lens, 1)),
        "out": (new(), lambda x: st.st_kv_attend(cache, new(), table, start, lens, 1, out=x)),
        "logits": (torch.zeros(2, 3, 50), lambda x: st.st_beam_select(x, torch.zeros(2, 3), 4)),
        "scores": (torch.zeros(2, 3), lambda x: st.st_beam_select(torch.zeros(2, 3, 50), x, 4)),
        "state 0": (torch.zeros(2, 3, 8), lambda x: st.st_beam_reorder([x], parents)),
        "out 0": (torch.zeros(2, 3, 8), lambda x: st.st_beam_reorder([torch.zeros(2, 3, 8)], parents, out=[x])),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_tensors_that_require_a_gradient(name):
    x, call = calls()[name]
    for tensor in (x.clone().requires_grad_(), x.clone().requires_grad_() * 2):
        with pytest.raises(ValueError, match=f"{name} requires a gradient"):
            call(tensor)
        for now in (lambda: call(tensor.detach()), lambda: torch.no_grad()(call)(tensor), lambda: torch.inference_mode()(call)(tensor)):
            with pytest.raises((ValueError, st.StError)) as e:  # the host's memory
                now()
            assert "gradient" not in str(e.value)
