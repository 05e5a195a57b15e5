"""The example network with texts that wait: the logits of a step belong to
the texts with new tokens, and steps that the cache has no room for are refused."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUND = 23 * 2.0 ** -8  # as in test_gpu_generate_example.py: 23 roundings to bf16 in a row


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__._libbuild().build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import generate
    return generate


def test_rows_of_the_texts_with_new_tokens(ex):
    assert ex.last_rows([[1], [2, 3], [4]]) == [0, 2, 3]
    assert ex.last_rows([[], [2, 3], [], [4], []]) == [1, 2]
    assert ex.last_rows([[], []]) == []


@pytest.mark.gpu
def test_waiting_texts(ex):
    model = ex.Model(ex.Config())
    g = torch.Generator().manual_seed(5)
    texts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in (3, 21, 40)]
    run = ex.Runner(model, 64, 3)
    done = [0, 0, 0]
    # the first text waits, then the second, then all but one; at last all go on
    for take in ((0, 20, 33), (2, 0, 1), (0, 0, 5), (1, 1, 1)):
        new = [t[d:d + n] for t, d, n in zip(texts, done, take)]
        done = [d + n for d, n in zip(done, take)]
        got = run.step(new)
        want = torch.cat([ex.reference(model, t[:d]) for t, d, n in zip(texts, done, take) if n])
        assert got.shape == want.shape
        off = ((got - want).norm(dim=1) / want.norm(dim=1)).max()
        assert float(off) <= BOUND


@pytest.mark.gpu
def test_steps_that_are_refused(ex):
    model = ex.Model(ex.Config(layers=1))
    run = ex.Runner(model, 16, 2)
    for new in ([[], []], [[1]], [[1], [2] * 17]):
        with pytest.raises(ValueError):
            run.step(new)
    with pytest.raises(ValueError):
        ex.generate(model, [[1, 2], []], 1)
