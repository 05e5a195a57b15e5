"""GPU tests of mt_tree_layout against parents followed one by one."""
import pytest
import torch

from tree_util import ancestors, bit_rows, mixed_tree, seen_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    return m


def check(mt, trees, words, kv=None, pad=0, lead=0, tail=0, stream=None, seen=None):
    """lead and tail rows belong to no sequence; visible's rows lie words + pad apart."""
    starts = [lead]
    for t in trees:
        starts.append(starts[-1] + len(t))
    T = starts[-1] + tail
    i32 = dict(dtype=torch.int32, device="cuda")
    parent = torch.full((T,), 12345, **i32)
    parent[lead:T - tail] = torch.tensor([p for t in trees for p in t], **i32)
    kv = kv or [len(t) + 100 + 7 * b for b, t in enumerate(trees)]
    positions = torch.full((T,), 77, **i32)
    store = torch.full((T, words + pad), 77, **i32)
    visible = store[:, :words]
    torch.cuda.synchronize()
    mt.mt_tree_layout(parent, torch.tensor(starts, **i32), torch.tensor(kv, **i32), positions, visible, stream=stream)
    torch.cuda.synchronize()
    seen = seen or [seen_of(t) for t in trees]
    want = torch.full((T, words), 77, dtype=torch.int32)
    want[lead:T - tail] = bit_rows(seen, T - tail - lead, words)
    place = torch.full((T,), 77, dtype=torch.int64)
    place[lead:T - tail] = torch.cat([kv[b] - len(t) + m.sum(1) - 1 for b, (t, m) in enumerate(zip(trees, seen))])
    assert torch.equal(visible.cpu(), want)
    assert torch.equal(positions.cpu().long(), place)
    assert bool((store[:, words:] == 77).all())


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 300, 1000, 1024])
def test_one_tree(mt, n):
    words = (n + 31) // 32
    check(mt, [mixed_tree(n, n)], words)
    check(mt, [list(range(-1, n - 1))], words)                  # a chain
    check(mt, [[-1] + [0] * (n - 1)], words)                    # a star
    check(mt, [[-1] * n], words)                                # no tree at all
    check(mt, [[(i - 1) // 3 if i else -1 for i in range(n)]], words)


def test_ragged_trees_with_rows_of_no_sequence(mt):
    trees = [mixed_tree(n, n, roots=1 + n % 3) for n in (5, 1, 0, 70, 33, 0, 128, 2)]
    check(mt, trees, 4, lead=3, tail=5)
    check(mt, trees, 9, pad=3)


def test_parents_that_are_not_earlier_tokens(mt):
    tree = [0, 5, 1, 3, -7, 4, 2 ** 31 - 1, -2 ** 31, 6, 9]
    m = seen_of(tree)
    assert int(m[1].sum()) == 1 and int(m[2].sum()) == 2 and int(m[8].sum()) == 2
    check(mt, [tree, mixed_tree(40, 3)], 2)


@pytest.mark.parametrize("n", [1025, 1500, 3001])
def test_more_tokens_than_bits(mt, n):
    # positions count every ancestor, the words hold the first 32 * words tokens
    for tree in (mixed_tree(n, n), list(range(-1, n - 1)), [max(-1, i - 40) for i in range(n)]):
        m = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):
            if tree[i] >= 0:
                m[i] = m[tree[i]]
            m[i, i] = True
        check(mt, [tree, mixed_tree(20, 1)], 32, seen=[m, seen_of(mixed_tree(20, 1))])
        check(mt, [tree], 3, seen=[m])


def test_many_trees(mt):
    check(mt, [mixed_tree(b % 23, b) for b in range(1024)], 1)


def test_either_output_alone_and_no_lengths(mt):
    tree = mixed_tree(1300, 5)
    i32 = dict(dtype=torch.int32, device="cuda")
    parent, start = torch.tensor(tree, **i32), torch.tensor([0, 1300], **i32)
    positions, visible = torch.zeros(1300, **i32), torch.zeros(1300, 32, **i32)
    mt.mt_tree_layout(parent, start, positions=positions)
    mt.mt_tree_layout(parent, start, visible=visible)
    assert positions.tolist() == [len(ancestors(tree, i)) - 1 for i in range(1300)]
    assert torch.equal(visible.cpu(), bit_rows([seen_of(tree)], 1300, 32))


def test_starts_beyond_the_rows_are_clamped(mt):
    i32 = dict(dtype=torch.int32, device="cuda")
    positions, visible = torch.full((40,), 9, **i32), torch.full((40, 2), 9, **i32)
    mt.mt_tree_layout(torch.tensor(mixed_tree(40, 2), **i32), torch.tensor([-5, 40, 30, 2000], **i32), torch.tensor([50, 7, 60], **i32), positions, visible)
    # [0, 40), nothing, [30, 40): the last sequence's rows are the first one's too, either may write them
    assert positions[:30].tolist() == [9 + len(ancestors(mixed_tree(40, 2), i)) for i in range(30)]


def test_other_stream_and_graph(mt):
    tree = mixed_tree(90, 6)
    check(mt, [tree], 3, stream=torch.cuda.Stream())
    i32 = dict(dtype=torch.int32, device="cuda")
    parent, start, kv = torch.zeros(90, **i32), torch.tensor([0, 90], **i32), torch.tensor([90], **i32)
    positions, visible = torch.zeros(90, **i32), torch.zeros(90, 3, **i32)
    graph = torch.cuda.CUDAGraph()
    mt.mt_tree_layout(parent, start, kv, positions, visible)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mt.mt_tree_layout(parent, start, kv, positions, visible)
    parent.copy_(torch.tensor(tree))
    kv.fill_(500)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(visible.cpu(), bit_rows([seen_of(tree)], 90, 3))
    assert positions.tolist() == [410 + len(ancestors(tree, i)) - 1 for i in range(90)]
