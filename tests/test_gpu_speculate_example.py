"""The example with drafted tokens: the logits along the accepted paths against
the same network in plain fp32 operations on the text alone, and the texts."""
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
    import speculate
    return speculate


def test_trees(ex):
    assert ex.tree_of((3,)) == ([-1, 0, 0, 0], [0, 1, 4])
    assert ex.tree_of((2, 2, 1)) == ([-1, 0, 0, 1, 1, 2, 2, 3, 4, 5, 6], [0, 1, 3, 7, 11])
    assert ex.tree_of((1, 1)) == ([-1, 0, 1], [0, 1, 2, 3])


def test_refusals(ex):
    for kw in (dict(prompts=[[1], []]), dict(tokens=0), dict(widths=()), dict(widths=(2, 0)), dict(drawn=True)):
        with pytest.raises(ValueError):
            ex.generate(type("M", (), {"cfg": ex.Config()})(), **{**dict(prompts=[[1]], tokens=3), **kw})


@pytest.mark.gpu
@pytest.mark.parametrize("widths", [(3, 2, 1), (1, 1, 1, 1, 1), (6, 3, 2)], ids=["tree", "chain", "55 tokens"])
@pytest.mark.parametrize("temperature,drawn", [(0.0, False), (0.8, False), (0.8, True)], ids=["greedy", "chosen", "drawn"])
def test_logits_and_texts(ex, widths, temperature, drawn):
    ex.mt.mt_device_error(True)
    model = ex.Model(ex.Config())
    for layer in model.layers:  # so that the draft, which has no layers, is often right
        layer["o"] *= 0.25
        layer["down"] *= 0.25
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in (1, 19, 70)]
    texts, raw = ex.generate(model, prompts, 12, temperature, widths, drawn, seed=4)
    assert ex.mt.mt_device_error(True) == 0
    if not drawn:  # some drafted tokens were accepted: more tokens of a text than steps
        assert sum(b == 0 for b, _, _ in raw) > len({id(l._base) for b, _, l in raw if b == 0})
    # every token of every text comes from one step, in order
    assert sorted((b, n) for b, n, _ in raw) == [(b, n) for b, (p, t) in enumerate(zip(prompts, texts)) for n in range(len(p), len(t))]
    for b, n, logits in raw:
        assert 12 <= len(texts[b]) - len(prompts[b]) <= 12 + len(widths)
        if temperature == 0:
            assert texts[b][n] == int((logits == logits.max()).nonzero()[0])  # the network's own choice
    # a step that follows accepted tokens, whose keys were moved, sees the text alone
    for b, n, logits in raw[-6:] + raw[:3]:
        want = ex.reference(model, texts[b][:n])[0]
        assert float((logits - want).norm() / want.norm()) <= BOUND


@pytest.mark.gpu
def test_window(ex):
    model = ex.Model(ex.Config(window=24, sinks=3))
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in (40, 9)]
    texts, raw = ex.generate(model, prompts, 10, 0.0, (2, 2, 1))
    for b, n, logits in raw[-5:]:
        want = ex.reference(model, texts[b][:n])[0]
        assert float((logits - want).norm() / want.norm()) <= BOUND
