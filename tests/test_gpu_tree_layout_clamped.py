"""GPU test of mt_tree_layout with starts outside the rows: both outputs, and
what lies behind them."""
import pytest
import torch

from tree_util import ancestors, bit_rows, mixed_tree, seen_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    return m


@pytest.mark.parametrize("words,pad", [(2, 0), (2, 1), (4, 0), (8, 8)])
def test_starts_beyond_the_rows(mt, words, pad):
    i32 = dict(dtype=torch.int32, device="cuda")
    T, guard = 40, 24
    tree = mixed_tree(T, 2)
    parent = torch.full((T + guard,), 0, **i32)
    parent[:T] = torch.tensor(tree, **i32)
    positions, store = torch.full((T + guard,), 9, **i32), torch.full((T + guard, words + pad), 9, **i32)
    mt.mt_tree_layout(parent[:T], torch.tensor([-5, 40, 30, 2000], **i32), torch.tensor([50, 7, 60], **i32), positions[:T], store[:T, :words])
    positions, store = positions.cpu(), store.cpu()
    assert bool((positions[T:] == 9).all()) and bool((store[T:] == 9).all()) and bool((store[:, words:] == 9).all())
    # [0, 40) of 50 tokens, nothing, [30, 40) of 60: rows 30 on belong to two sequences, either may write them
    first = [10 + len(ancestors(tree, i)) - 1 for i in range(T)]
    bits = bit_rows([seen_of(tree)], T, words)
    assert positions[:30].tolist() == first[:30]
    assert torch.equal(store[:30, :words], bits[:30])
    # the last sequence's parents are indices among its own ten tokens
    own = tree[30:40]
    second = [50 + len(ancestors(own, i)) - 1 for i in range(10)]
    own_bits = bit_rows([seen_of(own)], 10, words)
    for i in range(10):
        assert int(positions[30 + i]) in (first[30 + i], second[i])
        row = store[30 + i, :words]  # stored in words, each by either
        assert bool(((row == bits[30 + i]) | (row == own_bits[i])).all())
