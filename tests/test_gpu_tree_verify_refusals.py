"""GPU tests of mt_tree_verify where S, the sum of R over a token's refused
children, grows past 256: many refused children, and rows of large sums."""
import pytest
import torch

from tree_util import verify_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    return m


def check(mt, stars, V, p, q, cols=3, pad=0):
    """stars: a sequence's children of its first token, as (token, random) pairs, behind
    that token's random number; all rows are p and q.  Results are equal to the definition's
    and returned."""
    starts = [0]
    for _, children in stars:
        starts.append(starts[-1] + 1 + len(children))
    T, B = starts[-1], len(stars)
    tokens = torch.tensor([x for _, c in stars for x in [0] + [t for t, _ in c]], dtype=torch.int32)
    random = torch.tensor([x for u, c in stars for x in [u] + [r for _, r in c]])
    parent = torch.tensor([x for _, c in stars for x in [-1] + [0] * len(c)], dtype=torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")

    def rows(x):
        store = torch.full((T, V + pad), 0.5, device="cuda")
        store[:, :V] = x.cuda()
        return store[:, :V]
    out, path, count = torch.full((B, cols), 99, **i32), torch.full((B, cols), 99, **i32), torch.full((B,), 99, **i32)
    target, draft = p.expand(T, V), q.expand(T, V)
    mt.mt_tree_verify(rows(target), tokens.cuda(), parent.cuda(), random.cuda(), torch.tensor(starts, **i32), out, path, count, draft=rows(draft))
    want = verify_ref(target, draft, tokens, parent, random, starts, cols)
    got = out.tolist(), path.tolist(), count.tolist()
    assert got[2] == want[2]
    assert got[1] == want[1]
    assert got[0] == want[0]
    return want


@pytest.mark.parametrize("n", [340, 341, 342, 700])
def test_children_that_the_target_has_refused(mt, n):
    # R is 3/4 from the first refusal on: S is 256 after 341 of them.  Token 0 has nothing left then,
    # be it a child's or the draw's
    p, q = torch.tensor([0.25, 0.75]), torch.tensor([1.0, 0.0])
    refused = [(0, 0.9)] * n
    want = check(mt, [(u, refused + last) for u in (0.0, 0.1, 0.9) for last in ([], [(0, 0.1)], [(0, 0.0)], [(1, 0.5), (0, 0.1)])], 2, p, q)
    assert {t[0] for t in want[0]} == {1}


@pytest.mark.parametrize("pad", [0, 1], ids=["fours", "singles"])
@pytest.mark.parametrize("V", [60, 301])
def test_a_draft_that_shares_a_fifth_of_its_mass(mt, V, pad):
    # the target has 0.8 of its mass where the draft has none; 600 children are drawn from the
    # draft.  Entries are whole steps of 2^-12, so that the rational sums stay short
    g = torch.Generator().manual_seed(V)

    def row(n, mass):
        # `mass` / 4096 over n tokens, one at least each
        cut = torch.randint(0, n, (mass - n,), generator=g)
        return (torch.ones(n) + torch.bincount(cut, minlength=n)) / 4096
    half = V // 2
    p = torch.cat([row(half, 820), row(V - half, 3276)])
    q = torch.cat([row(half, 4096), torch.zeros(V - half)])
    stars = [(float(torch.rand(1, generator=g)), [(int(t), float(u)) for t, u in zip(torch.multinomial(q, 600, replacement=True, generator=g),
                                                                                    torch.rand(600, generator=g))])
             for _ in range(12 if V < 100 else 3)]
    # and one whose numbers refuse what can be refused
    stars.append((0.3, [(t, 1 - 2.0 ** -24) for t, _ in stars[0][1]]))
    check(mt, stars, V, p, q, pad=pad)


@pytest.mark.parametrize("pad", [0, 3], ids=["fours", "singles"])
@pytest.mark.parametrize("tail", [200, 4200])
def test_rows_of_large_sums(mt, tail, pad):
    # 16 tokens that only the draft has, `tail` that both do and 72 that only the target does: R is above
    # 36 all along, so that S passes 256 after some refusals; S q / p then decides over the tail
    own, both = 2.0 ** -5, 2.0 ** -9
    p = torch.cat([torch.zeros(16), torch.full((tail,), min(0.25, 64 / tail)), torch.full((72,), 0.5)])
    q = torch.cat([torch.full((16,), own), torch.full((tail,), both if tail < 1000 else both / 64), torch.zeros(72)])
    V = 88 + tail
    stars = []
    for k in (0, 1, 2, 3, 5, 7, 9, 12):  # k refused children, then one of the tail's
        for last in ([], [(16 + 3 * k, 0.5)], [(15 + tail, 0.999)]):
            for u in (0.0, 0.7):
                stars.append((u, [(i % 16, 0.5) for i in range(k)] + last))
    want = check(mt, stars, V, p, q, pad=pad)
    drawn = [t[0] for t in want[0]]
    assert any(t < 16 + tail for t in drawn) and any(t >= 16 + tail for t in drawn)
    assert {1, 2} == set(want[2])


def test_four_refused_in_rows_that_sum_to_a_hundred(mt):
    p = torch.cat([torch.full((200,), 0.5), torch.zeros(8)])
    q = torch.cat([torch.full((128,), 2.0 ** -8), torch.zeros(72), torch.full((8,), 2.0 ** -4)])
    for n in (1, 4, 8, 20):
        refused = [(200 + i % 8, 0.25) for i in range(n)]
        check(mt, [(u, refused + last) for u in (0.0, 0.3, 0.99) for last in ([], [(5, 0.0)], [(5, 0.9)], [(150, 0.9)])], 208, p, q)
