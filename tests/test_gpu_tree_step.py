"""The calls for drafted tokens one after another on several streams at a time,
without programmatic launch, and captured as one step into a graph."""
import math

import pytest
import torch

from paged_util import attention_bounds, check
from paged_util import Paged
from tree_util import bit_rows, mixed_tree, seen_of, tree_attention_ref, verify_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    m.mt_device_error(True)
    yield m
    assert m.mt_device_error(True) == 0


class Step:
    """A step of three texts: layout, attention, probabilities, verification, the kept tokens moved in two layers."""

    def __init__(self, mt, seed, V=9000, draft=False):
        self.mt, self.V = mt, V
        self.lens = [(25, 300), (1, 40), (60, 90)]
        self.trees = [mixed_tree(n, seed + b) for b, (n, _) in enumerate(self.lens)]
        p = self.p = Paged(self.lens, 8, 2, 64, page=16, seed=seed)
        self.q, self.k, self.v, self.pages, self.q_start, self.kv_len = p.cuda()
        g = torch.Generator().manual_seed(seed)
        T = p.T
        self.logits = torch.randn(T, V, generator=g) * 4
        drafted = self.logits + torch.randn(T, V, generator=g)
        self.tokens, self.random = torch.zeros(T, dtype=torch.int32), torch.rand(T, generator=g)
        self.parent = torch.tensor([x for t in self.trees for x in t], dtype=torch.int32)
        starts = self.starts = p.q_start.tolist()
        for a, t in zip(starts, self.trees):
            count = {}
            for i, up in enumerate(t):
                if up >= 0:
                    k = count[up] = count.get(up, 0) + 1
                    self.tokens[a + i] = int(drafted[a + up].topk(k).indices[-1])
        self.draft = torch.softmax(drafted, 1).cuda() if draft else None
        i32 = dict(dtype=torch.int32, device="cuda")
        self.dev = [x.cuda() for x in (self.logits, self.tokens, self.random, self.parent)]
        self.temperature = torch.full((T,), 0.8, device="cuda")
        self.positions, self.visible = torch.empty(T, **i32), torch.empty(T, 2, **i32)
        self.out, self.lse = torch.empty_like(self.q), torch.empty(T, 8, device="cuda")
        self.space = torch.empty(mt.mt_paged_attention_workspace_bytes(T, 3, 8, 2, 64), dtype=torch.uint8, device="cuda")
        self.probs = torch.empty(T, V, device="cuda")
        self.said, self.path = torch.empty(3, 6, **i32), torch.empty(3, 6, **i32)
        self.count, self.kept = torch.empty(3, **i32), torch.empty(3, **i32)
        self.layers = [(torch.randn_like(self.k), torch.randn_like(self.v)) for _ in range(2)]
        self.before = [(a.clone(), b.clone()) for a, b in self.layers]
        torch.cuda.synchronize()

    def run(self, stream=None):
        mt = self.mt
        logits, tokens, random, parent = self.dev
        mt.mt_tree_layout(parent, self.q_start, self.kv_len, self.positions, self.visible, stream=stream)
        mt.mt_tree_attention(self.q, self.k, self.v, self.pages, self.q_start, self.kv_len, self.visible, 60, 0.125, self.out, self.space,
                             lse=self.lse, stream=stream)
        mt.mt_token_probs(logits, self.probs, self.temperature, stream=stream)
        mt.mt_tree_verify(self.probs, tokens, parent, random, self.q_start, self.said, self.path, self.count, draft=self.draft, stream=stream)
        mt.mt_cache_keep(self.layers, self.pages, self.q_start, self.kv_len, self.path, self.count, new_len=self.kept, stream=stream)

    def compare(self):
        torch.cuda.synchronize()
        seen = [seen_of(t) for t in self.trees]
        assert torch.equal(self.visible.cpu(), bit_rows(seen, self.p.T, 2))
        ref = tree_attention_ref(self.p, seen, 0.125)
        tol_out, tol_lse = attention_bounds(self.p, ref, 2.0 ** -8, torch.bfloat16)
        check(self.out, ref[0], tol_out)
        check(self.lse, ref[1], tol_lse)
        said, path, count = verify_ref(self.probs.cpu(), self.draft.cpu() if self.draft is not None else None, self.tokens, self.parent,
                                       self.random, self.starts, 6)
        assert (self.said.tolist(), self.path.tolist(), self.count.tolist()) == (said, path, count)
        assert self.kept.tolist() == [kv - n + m for (n, kv), m in zip(self.lens, count)]
        for now, was in zip(self.layers, self.before):
            for x, y in zip(now, was):
                want = y.clone()
                for b, (n, kv) in enumerate(self.lens):
                    for i, at in enumerate(path[b][:count[b]]):
                        a, z = kv - n + at, kv - n + i
                        want[self.p.pages[b, z // 16], z % 16] = y[self.p.pages[b, a // 16], a % 16]
                assert torch.equal(x, want)
        return max(count)


@pytest.mark.parametrize("draft", [False, True], ids=["chosen", "drawn"])
def test_a_step(mt, draft):
    paths = []
    for seed in range(4):
        s = Step(mt, seed, draft=draft)
        s.run()
        paths.append(s.compare())
    assert max(paths) > 1


def test_steps_on_streams_at_a_time(mt):
    steps = [Step(mt, 10 + i, V=40000, draft=bool(i % 2)) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(2):  # what runs at the same time shares nothing
        for s, x in zip(streams, steps):
            for now, was in zip(x.layers, x.before):
                with torch.cuda.stream(s):
                    now[0].copy_(was[0])
                    now[1].copy_(was[1])
            x.run(stream=s)
    for x in steps:
        x.compare()


def test_without_programmatic_launch(mt):
    mt.mt_set_option(mt.MT_OPT_PDL, 0)
    try:
        s = Step(mt, 20, draft=True)
        s.run()
        s.compare()
    finally:
        mt.mt_set_option(mt.MT_OPT_PDL, 1)


def test_a_captured_step(mt):
    s, other = Step(mt, 30), Step(mt, 31)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    torch.cuda.synchronize()
    graph.replay()
    s.compare()
    # the same step with another's inputs
    for x, y in zip(s.dev + [s.q, s.k, s.v, s.pages], other.dev + [other.q, other.k, other.v, other.pages]):
        x.copy_(y)
    for (a, b), (c, d) in zip(s.layers, other.before):
        a.copy_(c)
        b.copy_(d)
    for name in ("p", "trees", "tokens", "random", "parent", "before"):
        setattr(s, name, getattr(other, name))
    graph.replay()
    s.compare()


def test_two_graphs_with_a_workspace_each(mt):
    a, b = Step(mt, 40), Step(mt, 41)
    graphs = []
    for x in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    a.compare()
    b.compare()
