"""The decode operators together, as one step after another of a beam decode
over the paged cache: eagerly against the plain forms, captured in a graph, and
on two streams at once."""
import math

import numpy as np
import pytest
import torch

import decode_ref as ref
import filtered_int8_ann_b200 as st

pytestmark = pytest.mark.gpu


class Decode:
    """One attention layer with random weights; B requests of K beams, the whole state in fixed buffers."""

    def __init__(self, seed, B=3, K=4, V=203, H=2, G=2, D=64, S=16, steps=40, prompt=(21, 5, 16), dtype=torch.bfloat16, end=7):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.B, self.K, self.V, self.H, self.G, self.D, self.S, self.end = B, K, V, H, G, D, S, end
        R, width = B * K, -(-(max(prompt) + steps) // S) + 1
        self.R, self.width, self.blocks = R, width, 2 * R * width
        self.dtype, m = dtype, 96
        self.embed = rnd(V, m)
        self.wq, self.wk, self.wv = rnd(m, H * G * D) / 6, rnd(m, H * D) / 10, rnd(m, H * D) / 10
        self.wo = rnd(H * G * D, V) / 2
        self.cache = st.KvCache.empty(self.blocks, H, S, D)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((R, width), -1, **i32)
        self.lens = torch.zeros(R, **i32)
        self.tokens = torch.zeros(R, dtype=torch.int64, device="cuda")
        self.scores = torch.full((B, K), -math.inf, device="cuda")
        self.scores[:, 0] = 0
        self.done = torch.zeros(B, K, dtype=torch.bool, device="cuda")
        self.history = torch.full((B, K, steps), -1, **i32)
        self.at = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.prompt = prompt

    def project(self, tokens):
        h = self.embed[tokens]
        heads = lambda x: x.view(len(tokens), -1, self.D).to(self.dtype)  # noqa: E731
        return heads(h @ self.wq), heads(h @ self.wk), heads(h @ self.wv)

    def attend(self, q, k, v, slots, sources, start, lens, most):
        st.st_kv_append(self.cache, k, v, slots, sources)
        return st.st_kv_attend(self.cache, q, self.table, start, lens, most, max_len=self.width * self.S)

    def choose(self, o, rows):
        logits = (o.flatten(1).float() @ self.wo)[rows].view(self.B, self.K, self.V)
        scores, parents, tokens, done = st.st_beam_select(logits, self.scores, self.K, finished=self.done, end_token=self.end)
        return logits, scores, parents, tokens, done

    def take(self, lens, scores, parents, tokens, done):
        B, K = self.B, self.K
        table, lens, history = st.st_beam_reorder([self.table.view(B, K, -1), lens.view(B, K), self.history], parents)
        self.table.copy_(table.view(self.R, -1))
        self.lens.copy_(lens.view(-1))
        self.history.copy_(history)
        self.history.scatter_(2, self.at.expand(B, K, 1), tokens[..., None])
        self.at += 1
        self.scores.copy_(scores)
        self.done.copy_(done)
        self.tokens.copy_(tokens.view(-1).clamp(min=0))

    def first(self):
        """The prompts go into each request's first beam, whose cache the others then share."""
        add = torch.zeros(self.R, dtype=torch.int32)
        add[::self.K] = torch.tensor(self.prompt, dtype=torch.int32)
        total = int(add.sum())
        tokens = torch.arange(total, device="cuda") * 37 % self.V
        slots, sources, start, lens, report = st.st_kv_plan(self.table, self.lens, add.cuda(), self.blocks, self.S, total)
        q, k, v = self.project(tokens)
        o = self.attend(q, k, v, slots, sources, start, lens, max(self.prompt))
        last = (start[1:].view(self.B, self.K)[:, :1] - 1).expand(self.B, self.K).reshape(-1).long()
        self.take(lens, *self.choose(o, last)[1:])
        return report

    def step(self):
        add = torch.ones_like(self.lens)
        slots, sources, start, lens, self.report = st.st_kv_plan(self.table, self.lens, add, self.blocks, self.S, self.R)
        q, k, v = self.project(self.tokens)
        o = self.attend(q, k, v, slots, sources, start, lens, 1)
        self.take(lens, *self.choose(o, torch.arange(self.R, device="cuda"))[1:])

    def state(self):
        return [x.clone() for x in (self.table, self.lens, self.history, self.scores, self.done, self.cache.k, self.cache.v,
                                    self.cache.k_scale, self.cache.v_scale)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,D,S", [(torch.bfloat16, 64, 16), (torch.float16, 128, 32)])
def test_steps_against_the_plain_forms(dtype, D, S):
    m = Decode(1, dtype=dtype, D=D, S=S)
    m.first()
    R, H = m.R, m.H
    host = [x.cpu().numpy().copy() for x in (m.cache.k, m.cache.v, m.cache.k_scale, m.cache.v_scale)]
    forked = False
    for step in range(30):
        table, have = m.table.cpu().tolist(), m.lens.tolist()
        add = [0 if step % 7 == 3 and r % 5 == 1 else 1 for r in range(R)]  # some rows wait for a step
        T = sum(add) + 2
        got = st.st_kv_plan(m.table, m.lens, torch.tensor(add, dtype=torch.int32).cuda(), m.blocks, S, T)
        want = ref.plan(table, have, add, m.blocks, S, T)
        assert m.table.cpu().tolist() == want[0]
        for x, y in zip(got, want[1:]):
            assert x.tolist() == list(y)
        slots, sources, start, lens, report = got
        assert report.tolist()[2:] == [0, 0]
        forked = forked or any(s >= 0 and s // S != src for s, src in zip(*[x.tolist() for x in (slots, sources)]))
        rows = torch.tensor([r for r in range(R) if add[r]] + [0, 0]).cuda()  # two padding tokens
        q, k, v = m.project(m.tokens[rows])
        o = m.attend(q, k, v, slots, sources, start, lens, 1)
        for i, x in enumerate((k, v)):
            ref.append(host[i], host[2 + i], x.float().cpu().numpy(), want[1], want[2])
        for x, y in zip((m.cache.k, m.cache.v, m.cache.k_scale, m.cache.v_scale), host):
            assert np.array_equal(x.cpu().numpy(), y)
        cpu = [torch.from_numpy(x) for x in host]
        wanted, parts = ref.attend(q.cpu(), cpu[0], cpu[1], cpu[2], cpu[3], want[0], want[3], want[4], D ** -0.5)
        n = sum(add)
        off = (o.cpu().double() - wanted).abs() - ref.attend_tolerance(wanted, parts, dtype, D)
        assert bool((off[:n] <= 0).all())
        place = torch.zeros(R, dtype=torch.int64)
        place[rows[:n].cpu()] = torch.arange(n)
        logits, scores, parents, tokens, done = m.choose(o, place.cuda())
        for b, pairs in enumerate(ref.select(logits.cpu(), m.scores.cpu(), m.K, finished=m.done.cpu(), end=m.end)):
            assert parents[b].tolist() == [p[1] for p in pairs] and tokens[b].tolist() == [p[2] for p in pairs]
        before = m.table.view(m.B, m.K, -1).clone(), lens.view(m.B, m.K).clone()
        m.take(lens, scores, parents, tokens, done)
        for b in range(m.B):
            assert torch.equal(m.table.view(m.B, m.K, -1)[b], before[0][b][parents[b].long()])
            assert torch.equal(m.lens.view(m.B, m.K)[b], before[1][b][parents[b].long()])
    assert forked, "no row ever got a block of its own for a shared one"
    assert st.st_decode_check() == st.ST_OK


def test_steps_captured_in_a_graph_repeat_the_eager_ones():
    eager, graphed = Decode(2, steps=60), Decode(2, steps=60)
    for m in (eager, graphed):
        m.first()
        for _ in range(3):  # eager steps first: limits raised, allocator warm
            m.step()
    assert same(eager.state(), graphed.state())
    for _ in range(40):
        eager.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        graphed.step()
    for _ in range(40):
        graph.replay()
    torch.cuda.synchronize()
    assert same(eager.state(), graphed.state())
    assert st.st_decode_check() == st.ST_OK


def test_two_decodes_on_two_streams():
    """Captured and eager steps of two decodes at once give what each gives alone."""
    alone = []
    for seed in (3, 4):
        m = Decode(seed, K=5, G=4)
        m.first()
        for _ in range(20):
            m.step()
        alone.append(m.state())
    both = [Decode(3, K=5, G=4), Decode(4, K=5, G=4)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    graphs = []
    for m, s in zip(both, streams):
        with torch.cuda.stream(s):
            m.first()
            m.step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            m.step()
        graphs.append(graph)
    for i in range(19):
        for m, s, graph in zip(both, streams, graphs):
            with torch.cuda.stream(s):
                if i % 3:
                    graph.replay()
                else:
                    m.step()
    torch.cuda.synchronize()
    for m, want in zip(both, alone):
        assert same(m.state(), want)


def test_calls_on_a_stream_given():
    """The stream argument: work and outputs belong to that stream, whatever the current one."""
    m = Decode(5)
    m.first()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = torch.randn(4, 3, 5000, device="cuda")
    scores = -torch.rand(4, 3, device="cuda")
    q = torch.randn(m.R, m.H * m.G, m.D, device="cuda").to(m.dtype)
    start = torch.arange(m.R + 1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    want = st.st_beam_select(x, scores, 6), st.st_kv_attend(m.cache, q, m.table, start, m.lens, 1), st.st_beam_reorder([x], torch.zeros(4, 2, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    p = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = st.st_beam_select(x, scores, 6, stream=stream), st.st_kv_attend(m.cache, q, m.table, start, m.lens, 1, stream=stream), st.st_beam_reorder([x], p, stream=stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[0][:3], want[0][:3]))
        assert torch.equal(got[1], want[1]) and torch.equal(got[2][0], want[2][0])


def test_results_repeat_bit_for_bit():
    g = torch.Generator(device="cuda").manual_seed(6)
    x = (3 * torch.randn(3, 8, 40001, generator=g, device="cuda")).bfloat16()
    s = -torch.rand(3, 8, generator=g, device="cuda")
    S, H, D, n = 32, 2, 128, 9000
    cache = st.KvCache(torch.randint(-127, 128, (300, H, S, D), generator=g, device="cuda", dtype=torch.int8), torch.randint(-127, 128, (300, H, S, D), generator=g, device="cuda", dtype=torch.int8),
                       torch.rand(300, H, generator=g, device="cuda"), torch.rand(300, H, generator=g, device="cuda"))
    table = torch.randperm(300, generator=g, device="cuda").int()[:290].view(1, -1).contiguous()
    for m in (1, 3, 200):
        q = torch.randn(m, 4 * H, D, generator=g, device="cuda").half()
        args = (q, table, torch.tensor([0, m], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda"), m)
        first = st.st_kv_attend(cache, *args)
        assert all(torch.equal(first, st.st_kv_attend(cache, *args)) for _ in range(5))
    first = st.st_beam_select(x, s, 50)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first[:3], st.st_beam_select(x, s, 50)[:3]))


def test_workspaces_given():
    """A workspace of the size asked for is enough; a smaller one is refused."""
    import ctypes
    m = Decode(7)
    m.first()
    need = ctypes.c_int64(0)
    x, s = torch.randn(2, 3, 20000, device="cuda"), -torch.rand(2, 3, device="cuda")
    assert st.lib().st_beam_select_workspace(2, 3, 20000, 4, ctypes.byref(need)) == st.ST_OK and need.value > 0
    room = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    a, b = st.st_beam_select(x, s, 4, workspace=room), st.st_beam_select(x, s, 4)
    assert all(torch.equal(i, j) for i, j in zip(a[:3], b[:3]))
    with pytest.raises(st.StError) as e:
        st.st_beam_select(x, s, 4, workspace=room[:-16])
    assert e.value.status == st.ST_ERR_INVALID_ARG
    S, H, D, n = 16, 1, 64, 3000
    cache = st.KvCache.empty(200, H, S, D)
    q = torch.randn(1, 2, D, device="cuda").half()
    args = (q, torch.arange(190, dtype=torch.int32, device="cuda").view(1, -1), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda"), 1)
    assert st.lib().st_kv_attend_workspace(ctypes.byref(cache._c), 1, 2, 1, 1, 190 * 16, ctypes.byref(need)) == st.ST_OK and need.value > 0
    room = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    assert bool((st.st_kv_attend(cache, *args, workspace=room) == 0).all())
    with pytest.raises(st.StError):
        st.st_kv_attend(cache, *args, workspace=room[:-16])
