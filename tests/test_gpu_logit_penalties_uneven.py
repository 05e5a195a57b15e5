"""GPU tests of mt_logit_penalties where a sequence has more tokens than its
table holds: ranges of the vocabulary, one after the other and shared out over
blocks, among sequences that take the table."""
import pytest
import torch

from paged_util import HALF, check
from test_gpu_logit_penalties import mt, ragged, reference, words  # noqa: F401  (mt: a fixture)

pytestmark = pytest.mark.gpu

# (vocabulary, histories): 2048 slots at least, four for an average token; a
# sequence with more than three quarters of them goes over ranges of the
# vocabulary.  25 ranges in one block each, in 7 blocks, 4 ranges in 16 blocks
# (some without one), and every sequence over 2 ranges.
CASES = {"one of 200": (50257, [6000] + [3 * (b % 70) for b in range(199)]),
         "two of 40": (50257, [20] * 7 + [6000] + [0] * 30 + [5000, 1]),
         "one of 2": (50257, [20000, 20]),
         "all of 3": (20011, [13000, 14000, 16001])}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("biases,in_place,mask", [(True, False, True), (True, True, False), (False, True, True), (False, False, False)],
                         ids=["biases-mask", "biases-in-place", "in-place-mask", "plain"])
def test_long_histories_among_short_ones(mt, name, dtype, biases, in_place, mask):  # noqa: F811
    V, lens = CASES[name]
    B = len(lens)
    g = torch.Generator().manual_seed(40)
    x = (torch.randn(B, V, generator=g) * 4).to(dtype)
    # frequent and rare tokens, and padding on both sides of the vocabulary
    hist = [(V * torch.rand(n, generator=g, dtype=torch.float64) ** 3).long().tolist() for n in lens]
    for h in hist:
        h[5::17] = [-1] * len(h[5::17])
        h[6::19] = [V + 2] * len(h[6::19])
        if len(h) > 4000:
            h[:4] = [0, V - 1, 2047, 2048]  # the ranges' ends
    prompt = [len(h) // 3 for h in hist]
    bias = [list(zip(torch.randint(0, V, (9,), generator=g).tolist() + [3, 3, V - 1], torch.randn(12, generator=g).tolist()))
            if biases else [] for _ in range(B)]
    rep, pres, freq = 1 + 0.4 * torch.rand(B, generator=g), torch.rand(B, generator=g), torch.rand(B, generator=g) * 0.1
    allowed = torch.rand(B, V, generator=g) < 0.7 if mask else None
    h, hs = ragged(hist, torch.int32)
    kw = dict(history=h, history_start=hs, prompt_len=torch.tensor(prompt, dtype=torch.int32), repetition=rep, presence=pres,
              frequency=freq)
    if biases:
        ids, bs = ragged([[t for t, _ in row] for row in bias], torch.int32)
        kw.update(bias_ids=ids, bias_start=bs, bias_values=torch.tensor([w for row in bias for _, w in row]))
    if mask:
        kw["allowed"] = words(allowed)
    src = x.cuda()
    dst = src if in_place else torch.full_like(src, 7.0)
    mt.mt_logit_penalties(src, dst, **{k: v.cuda() for k, v in kw.items()})
    want, size = reference(x, hist, prompt, rep.double(), pres.double(), freq.double(), bias, allowed)
    # bias sum, quotient or product, and two sums in fp32, then the output's rounding
    tol = HALF[dtype] * want.abs().nan_to_num(posinf=0) + 8 * 2.0 ** -24 * size + 1e-30
    check(dst, want, tol)
