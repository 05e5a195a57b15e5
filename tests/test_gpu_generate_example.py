"""The example that runs the library's calls as a whole network: its logits
against the same network in plain fp32 operations, and its texts' constraints."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A layer rounds to bf16 (2^-8 relative at most) after each of its ten tensors
# (two sums, two norms, q/k/v, their rotation, attention, o, h, y) and inside
# attention's weights; two layers and the last norm: 23 roundings in a row, of
# which each reaches the logits at most in proportion.
BOUND = 23 * 2.0 ** -8


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import generate
    import quantized_gemv_epilogues_gb300 as mt
    torch.cuda.set_device(0)
    mt.mt_device_error(True)
    yield generate
    assert mt.mt_device_error(True) == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_logits_and_texts(ex, window, sinks):
    model = ex.Model(ex.Config(window=window, sinks=sinks))
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in (1, 19, 70)]
    free, _ = ex.generate(model, prompts, 4)
    banned = free[0][len(prompts[0])]  # the first token that the first text takes
    texts, raw = ex.generate(model, prompts, 6, banned=banned)
    for p, t in zip(prompts, texts):
        assert len(t) == len(p) + 6 and t[:len(p)] == p and banned not in t[len(p):]
    for k in (0, 2, 5):
        want = torch.cat([ex.reference(model, t[:len(p) + k]) for p, t in zip(prompts, texts)])
        off = ((raw[k] - want).norm(dim=1) / want.norm(dim=1)).max()
        assert float(off) <= BOUND
