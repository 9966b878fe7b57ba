"""The documented beam decode step, run on stand-ins of the calls: which length goes with which table row, and what
happens when the pool has run out."""
import os
import re
import textwrap
import types

import pytest
import torch

import filtered_int8_ann_b200 as st
from filtered_int8_ann_b200 import decode

B, K, R, WIDTH = 2, 3, 6, 5
I32 = torch.int32


def readme_step():
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    step, = (b for b in blocks if "st_kv_plan" in b)
    return step


def docstring_step():
    lines = decode.__doc__.split("A step, for R rows", 1)[1].split("\n\n", 1)[1]
    return textwrap.dedent(re.match(r"(?:    .*\n|\n)+", lines).group(0))


def gather(states, parents):
    return [torch.stack([x[b, parents[b].long()] for b in range(B)]) for x in states]


def run(step, served):
    have = torch.tensor([7, 0, 0, 9, 9, 3], dtype=I32)
    lens, report = have + 1, torch.tensor([2, 9, 0, 0], dtype=I32)
    if not served:
        lens[4], report[2] = -1, 1
    table = torch.arange(R * WIDTH, dtype=I32).view(R, WIDTH)
    parents, tokens = torch.tensor([[1, 0, 0], [2, 0, 1]], dtype=I32), torch.zeros(B, K, dtype=I32)
    called = []

    def call(name, result):
        def f(*a, **k):
            called.append(name)
            return result(*a) if callable(result) else result
        return f

    calls = {"st_kv_plan": call("plan", (torch.zeros(R, dtype=torch.int64), torch.zeros(R, dtype=I32), torch.arange(R + 1, dtype=I32), lens, report)),
             "st_kv_append": call("append", None), "st_kv_attend": call("attend", torch.zeros(R, 4, 128)),
             "st_beam_select": call("select", (torch.zeros(B, K), parents, tokens, None)), "st_beam_reorder": call("reorder", gather),
             "st_decode_check": call("check", st.ST_OK)}
    ns = dict(calls, st=types.SimpleNamespace(**calls, KvCache=types.SimpleNamespace(empty=lambda *a: None), ST_OK=st.ST_OK), cache=None, table=table, have=have,
              add=torch.ones(R, dtype=I32), num_blocks=99, kv_heads=1, block_size=32, T=R, R=R, B=B, K=K, keep=K, max_q=1, q=None, k=None, v=None,
              longest=40, logits=torch.zeros(B, K, 11), scores=torch.zeros(B, K), seqs=torch.zeros(B, K, 2, dtype=I32))
    before = table.clone()
    try:
        exec(step, ns)
    finally:
        ns["called"] = called
        run.last = ns
    return ns, lens, gather([before.view(B, K, -1), lens.view(B, K)], parents)


@pytest.mark.parametrize("step", [readme_step, docstring_step])
def test_lengths_go_with_the_tables(step):
    ns, lens, (table, have) = run(step(), True)
    assert ns["called"][:4] == ["plan", "append", "attend", "select"] and "reorder" in ns["called"]
    assert torch.equal(ns["table"].reshape(R, -1), table.view(R, -1))
    assert torch.equal(ns["have"].reshape(R), have.view(R))


@pytest.mark.parametrize("step", [readme_step, docstring_step])
def test_rows_that_were_not_served_stop_the_step(step):
    """Their -1 is no length, and their tokens are not in the cache."""
    with pytest.raises(AssertionError):
        run(step(), False)
    assert run.last["called"] == ["plan"]
