"""GPU tests of mt_logit_penalties' lists: offsets of nearly 2^31 entries."""
import pytest
import torch

from test_gpu_logit_penalties import mt  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["history", "bias"])
def test_lists_that_end_at_the_last_32_bit_offset(mt, which):  # noqa: F811
    # the only sequence's entries are the last 5000 of 2^31 - 1
    n, own, V = 2 ** 31 - 1, 5000, 20011
    g = torch.Generator().manual_seed(9)
    ids = torch.randint(0, V, (own,), generator=g)
    flat = torch.empty(n, dtype=torch.int32, device="cuda")
    flat[n - own:] = ids.to(torch.int32).cuda()
    start = torch.tensor([n - own, n], dtype=torch.int32, device="cuda")
    x = torch.randn(1, V, generator=g)
    out = torch.empty(1, V, device="cuda")
    want = x.clone()
    if which == "history":
        one = torch.ones(1, device="cuda")
        mt.mt_logit_penalties(x.cuda(), out, history=flat, history_start=start, frequency=one)
        want[0] -= torch.bincount(ids, minlength=V).float()
    else:
        values = torch.empty(n, device="cuda")
        values[n - own:] = 1.0 + torch.arange(own, device="cuda")
        mt.mt_logit_penalties(x.cuda(), out, bias_ids=flat, bias_values=values, bias_start=start)
        last = {int(t): 1.0 + i for i, t in enumerate(ids)}
        want[0, list(last)] += torch.tensor(list(last.values()))
    assert torch.equal(out.cpu(), want)
