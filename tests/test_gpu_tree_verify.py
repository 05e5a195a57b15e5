"""GPU tests of mt_tree_verify against the definition in rationals: accepted
paths and drawn tokens have to be equal."""
import math

import pytest
import torch

from tree_util import mixed_tree, verify_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    return m


class Case:
    """Trees with a target's and a draft's rows: q is a coarser p, tokens come
    from q (drawn, or its largest)."""

    def __init__(self, trees, V, draft, seed=0, scale=3.0, noise=1.0, lead=0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.starts = [lead]
        for t in trees:
            self.starts.append(self.starts[-1] + len(t))
        self.T, self.V = self.starts[-1] + tail, V
        x = torch.randn(self.T, V, generator=g) * scale
        self.target = torch.softmax(x, 1)
        q = torch.softmax(x + torch.randn(self.T, V, generator=g) * noise, 1)
        self.draft = q if draft else None
        self.parent = torch.full((self.T,), -1, dtype=torch.int32)
        self.tokens = torch.zeros(self.T, dtype=torch.int32)
        self.random = torch.rand(self.T, generator=g)
        for a, tree in zip(self.starts, trees):
            count = {}
            for i, p in enumerate(tree):
                self.parent[a + i] = p
                if 0 <= p < i:
                    k = count[p] = count.get(p, 0) + 1
                    if draft:
                        self.tokens[a + i] = int(torch.multinomial(q[a + p], 1, generator=g))
                    else:
                        self.tokens[a + i] = int(torch.topk(q[a + p], min(k, V)).indices[-1])

    def run(self, mt, cols, pad=0, stream=None):
        T, V, B = self.T, self.V, len(self.starts) - 1
        i32 = dict(dtype=torch.int32, device="cuda")

        def rows(x):
            if x is None:
                return None
            store = torch.full((T, V + pad), math.nan, device="cuda")
            store[:, :V] = x.cuda()
            return store[:, :V]
        out, path, count = torch.full((B, cols), 99, **i32), torch.full((B, cols), 99, **i32), torch.full((B,), 99, **i32)
        args = [rows(self.target), self.tokens.cuda(), self.parent.cuda(), self.random.cuda(), torch.tensor(self.starts, **i32), out, path, count]
        draft = rows(self.draft)
        torch.cuda.synchronize()
        mt.mt_tree_verify(*args, draft=draft, stream=stream)
        torch.cuda.synchronize()
        return out.tolist(), path.tolist(), count.tolist()

    def check(self, mt, cols=8, **kw):
        got = self.run(mt, cols, **kw)
        want = verify_ref(self.target, self.draft, self.tokens, self.parent, self.random, self.starts, cols)
        assert got[2] == want[2]
        assert got[1] == want[1]
        assert got[0] == want[0]
        return want


def chain(n):
    return list(range(-1, n - 1))


DRAFT = pytest.mark.parametrize("draft", [False, True], ids=["chosen", "drawn"])


@DRAFT
@pytest.mark.parametrize("V", [1, 2, 5, 31, 32, 33, 100, 1000, 4097])
def test_vocabularies(mt, draft, V):
    c = Case([chain(5), mixed_tree(9, 1), [-1], [-1, 0, 0, 0, 1, 1, 2]] * 4, V, draft, seed=V)
    depths = {n for n in c.check(mt)[2]}
    assert V < 5 or len(depths) > 1


@DRAFT
@pytest.mark.parametrize("V", [20011, 50257])
def test_large_vocabularies(mt, draft, V):
    Case([chain(4), mixed_tree(8, 1), [-1]], V, draft, seed=V, scale=2.0).check(mt)


@DRAFT
@pytest.mark.parametrize("n", [1, 2, 31, 33, 60, 130, 300])
def test_tree_sizes(mt, draft, n):
    trees = [mixed_tree(n, n), chain(n), [-1] + [0] * (n - 1), [(i - 1) // 3 if i else -1 for i in range(n)]]
    # a draft that is nearly the target, so that paths are long; and one that is not
    Case(trees, 60, draft, seed=n, scale=4.0, noise=0.1).check(mt, cols=12)
    Case(trees, 60, draft, seed=n, noise=4.0).check(mt, cols=12)


@pytest.mark.parametrize("n", [1100, 2500])
def test_trees_of_many_tokens(mt, n):
    wide = [-1] + [0] * 40 + [1 + i % 40 for i in range(n - 41)]
    c = Case([wide, mixed_tree(n, 2)], 50, False, seed=n, scale=0.5, noise=4.0)
    c.check(mt, cols=6)
    c = Case([chain(n)], 7, True, seed=3, scale=3.0, noise=0.0)
    assert c.check(mt, cols=2000)[2][0] == min(n, 2000)  # the draft is the target: everything is accepted


@DRAFT
@pytest.mark.parametrize("cols", [1, 2, 3, 40])
def test_columns(mt, draft, cols):
    Case([chain(6), mixed_tree(20, 4)] * 6, 40, draft, seed=cols, scale=4.0, noise=0.2).check(mt, cols=cols)


@DRAFT
def test_sequences_without_tokens_and_rows_of_none(mt, draft):
    Case([[], chain(4), [], [], mixed_tree(12, 2), []], 90, draft, seed=3, lead=2, tail=3).check(mt)


@DRAFT
def test_strides(mt, draft):
    for pad in (1, 2, 3, 4, 64):
        Case([chain(4), mixed_tree(11, 2)], 131, draft, seed=pad).check(mt, pad=pad)
        Case([chain(4), mixed_tree(11, 2)], 4200, draft, seed=pad).check(mt, pad=pad)


@DRAFT
def test_many_sequences(mt, draft):
    Case([mixed_tree(1 + b % 7, b) for b in range(1024)], 23, draft, seed=5).check(mt)


@DRAFT
def test_the_same_token_twice(mt, draft):
    # siblings of one token: refused once, it has nothing left without a draft, and less with one
    c = Case([[-1] + [0] * 6 + [1, 2, 3]] * 40, 6, draft, seed=6, scale=1.0)
    for a in c.starts[:-1]:
        c.tokens[a + 1:a + 7] = torch.tensor([2, 2, 4, 2, 4, 1])
    c.check(mt)


@DRAFT
def test_numbers_at_their_ends(mt, draft):
    for u in (0.0, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan, math.inf, 2.0 ** -30, 2.0 ** -60):
        c = Case([chain(4), mixed_tree(9, 2), [-1]] * 3, 50, draft, seed=7)
        c.random[:] = u
        c.check(mt)
        c.random[::2] = 0.5
        c.check(mt)


@DRAFT
def test_equality_is_a_refusal(mt, draft):
    # probabilities and numbers in eighths: random q R = r exactly, and running sums that meet the number
    g = torch.Generator().manual_seed(8)
    trees = [[-1, 0, 0, 0, 1, 1], chain(4)] * 60
    c = Case(trees, 8, draft, seed=8)

    def eighths():
        p = torch.zeros(c.T, 8)
        p.scatter_add_(1, torch.randint(0, 8, (c.T, 8), generator=g), torch.full((c.T, 8), 0.125))
        return p
    c.target = eighths()
    if draft:
        c.draft = eighths()
    c.tokens = torch.randint(0, 8, (c.T,), generator=g).to(torch.int32)
    c.random = torch.randint(0, 8, (c.T,), generator=g) / 8.0
    c.check(mt)


@DRAFT
def test_rows_of_one_token(mt, draft):
    # a temperature of 0: what is drafted right is accepted, the first that is not is replaced
    g = torch.Generator().manual_seed(9)
    c = Case([chain(5), mixed_tree(15, 3)] * 10, 30, draft, seed=9)
    best = torch.randint(0, 30, (c.T,), generator=g)
    c.target = torch.nn.functional.one_hot(best, 30).float()
    for a, z in zip(c.starts[:-1], c.starts[1:]):
        for i in range(1, z - a):
            if int(torch.randint(0, 3, (1,), generator=g)):
                c.tokens[a + i] = best[a + int(c.parent[a + i])]
    want = c.check(mt)
    assert max(want[2]) > 2


@DRAFT
def test_rows_that_are_no_probabilities(mt, draft):
    # zeros, NaN, negative entries and ones above 1; sums of other than 1; a row without any mass draws -1
    g = torch.Generator().manual_seed(10)
    c = Case([chain(3), mixed_tree(9, 1), [-1], [-1, 0, 0]] * 8, 40, draft, seed=10)
    c.target[torch.rand(c.T, 40, generator=g) < 0.1] = math.nan
    c.target[torch.rand(c.T, 40, generator=g) < 0.1] = -1.0
    c.target[torch.rand(c.T, 40, generator=g) < 0.1] = 3.0
    c.target[torch.rand(c.T, 40, generator=g) < 0.1] = math.inf
    c.target[torch.rand(c.T, generator=g) < 0.3] = 0.0
    if draft:
        c.draft[torch.rand(c.T, 40, generator=g) < 0.1] = math.nan
        c.draft[torch.rand(c.T, generator=g) < 0.2] = 0.0
    assert any(-1 in t[:n] for t, _, n in zip(*c.check(mt)))


@DRAFT
def test_tokens_outside_the_vocabulary_are_refused(mt, draft):
    c = Case([[-1, 0, 0, 0, 1, 2, 3]] * 20, 30, draft, seed=11, noise=0.1)
    for a in c.starts[:-1]:
        c.tokens[a + 1], c.tokens[a + 4] = -1, 30
        c.tokens[a + 2] = 2 ** 31 - 1
    c.check(mt)


@DRAFT
def test_parents_that_are_not_earlier_tokens(mt, draft):
    # tokens below none are never reached, whatever hangs on them
    c = Case([[-1, 0, -1, 2, 1, 3, 0]] * 20, 30, draft, seed=12, scale=4.0, noise=0.1)
    c.check(mt)
    c.parent[2::7] = 100
    c.parent[5::7] = 6
    c.check(mt)


@DRAFT
def test_rows_of_leaves_may_be_anything(mt, draft):
    c = Case([chain(4)] * 10, 30, draft, seed=13)
    want = c.check(mt)
    if draft:
        for a in c.starts[1:]:
            c.draft[a - 1] = math.nan
        assert c.check(mt) == want


@DRAFT
def test_rows_further_apart_than_32_bits(mt, draft):
    far, V = (1 << 30) + 3, 3000
    c = Case([chain(4)], V, draft, seed=14, noise=0.1)
    i32 = dict(dtype=torch.int32, device="cuda")

    def rows(x):
        store = torch.empty(3 * far + V, device="cuda").as_strided((4, V), (far, 1))
        store.copy_(x)
        return store
    out, path, count = torch.zeros(1, 5, **i32), torch.zeros(1, 5, **i32), torch.zeros(1, **i32)
    mt.mt_tree_verify(rows(c.target), c.tokens.cuda(), c.parent.cuda(), c.random.cuda(), torch.tensor(c.starts, **i32), out, path, count,
                      draft=rows(c.draft) if draft else None)
    assert (out.tolist(), path.tolist(), count.tolist()) == verify_ref(c.target, c.draft, c.tokens, c.parent, c.random, c.starts, 5)


@pytest.mark.parametrize("shape", ["chain", "star", "tree"])
@DRAFT
def test_tokens_are_distributed_as_the_target(mt, draft, shape):
    """The first and second tokens over 1024 * 40 draws, whose counts are within five standard
    deviations of the target's probabilities."""
    B, V, rounds = 1024, 4, 40
    tree = {"chain": [-1, 0, 1], "star": [-1, 0, 0, 0], "tree": [-1, 0, 0, 1, 2]}[shape]
    n = len(tree)
    g = torch.Generator(device="cuda").manual_seed(15)
    p, q = torch.tensor([0.5, 0.25, 0.15, 0.1], device="cuda"), torch.tensor([0.2, 0.2, 0.5, 0.1], device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    target, drafts = p.expand(B * n, V).contiguous(), q.expand(B * n, V).contiguous()
    out, path, count = torch.zeros(B, 4, **i32), torch.zeros(B, 4, **i32), torch.zeros(B, **i32)
    starts, parent = torch.arange(0, B * n + 1, n, **i32), torch.tensor(tree * B, **i32)
    seen, second, met = torch.zeros(V, device="cuda"), torch.zeros(V, device="cuda"), 0
    for _ in range(rounds):
        if draft:
            tokens = torch.multinomial(q.expand(B * n, V), 1, generator=g)[:, 0].to(torch.int32)
        else:
            tokens = torch.tensor([[0, 2, 1, 3, 0][i] for i in range(n)] * B, **i32)
        mt.mt_tree_verify(target, tokens, parent, torch.rand(B * n, generator=g, device="cuda"), starts, out, path, count,
                          draft=drafts if draft else None)
        seen += torch.bincount(out[:, 0], minlength=V)
        two = out[count > 1][:, 1]
        second += torch.bincount(two, minlength=V)
        met += two.numel()
    for got, total in ((seen, B * rounds), (second, met)):
        off = (got.double() - total * p.double()).abs() / (total * p.double() * (1 - p.double())).sqrt()
        assert float(off.max()) < 5, (got / total).tolist()


@DRAFT
def test_other_stream_graph_and_equal_runs(mt, draft):
    c = Case([chain(5), mixed_tree(30, 3)] * 8, 5000, draft, seed=16)
    want = c.check(mt, stream=torch.cuda.Stream())
    assert c.run(mt, 8) == want
    i32 = dict(dtype=torch.int32, device="cuda")
    B = len(c.starts) - 1
    out, path, count = torch.zeros(B, 8, **i32), torch.zeros(B, 8, **i32), torch.zeros(B, **i32)
    ins = [c.target.cuda(), c.tokens.cuda(), c.parent.cuda(), c.random.cuda(), torch.tensor(c.starts, **i32)]
    q = c.draft.cuda() if draft else None
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mt.mt_tree_verify(*ins, out, path, count, draft=q)
    graph.replay()
    torch.cuda.synchronize()
    assert (out.tolist(), path.tolist(), count.tolist()) == want
    c.random = 1 - c.random
    ins[3].copy_(c.random)
    graph.replay()
    torch.cuda.synchronize()
    assert (out.tolist(), path.tolist(), count.tolist()) == verify_ref(c.target, c.draft, c.tokens, c.parent, c.random, c.starts, 8)
