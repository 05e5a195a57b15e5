"""GPU tests of mt_logit_penalties' arithmetic, operation by operation: each is
one fp32 operation, rounded to nearest, as the header writes it."""
import math

import pytest
import torch

from test_gpu_logit_penalties import mt  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def call(mt, x, out, **kw):
    """Every token is in the history once, so that all of them are penalised."""
    B, V = x.shape
    up = {k: torch.as_tensor(v, dtype=torch.float32).cuda() for k, v in kw.items()}
    mt.mt_logit_penalties(x.cuda(), out, history=torch.arange(V, dtype=torch.int32).repeat(B).cuda(),
                          history_start=(torch.arange(B + 1) * V).to(torch.int32).cuda(), **up)
    return out.cpu()


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_repetition_is_a_quotient(mt, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(1)
    # 2^-140 and 3e-39: reciprocals that fp32 does not hold
    rep = [1.3, 3.0, 0.7, 1e30, 1e-30, 2.0 ** -140, 3e-39, math.inf]
    x = torch.randn(len(rep), 3001, generator=g) * 10
    x[5:7] *= 2.0 ** -139
    x[:, 0], x[:, 1], x[:, 2] = 0.0, math.inf, -math.inf
    x = x.to(dtype)
    got = call(mt, x, torch.empty_like(x, device="cuda"), repetition=rep)
    r = torch.tensor(rep)[:, None]
    y = x.float()
    want = torch.where(y > 0, y / r, y * r).to(dtype)
    assert same(got, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_frequency_and_presence_are_added_first(mt, dtype):  # noqa: F811
    # terms that cancel, beside which the logit would be lost; and one that is not finite
    x = (torch.randn(4, 777, generator=torch.Generator().manual_seed(2)) * 4).to(dtype)
    freq, pres = [2.0 ** 100, -(2.0 ** 60), 0.5, math.inf], [-(2.0 ** 100), 2.0 ** 60, 0.25, 1.0]
    got = call(mt, x, torch.empty_like(x, device="cuda"), frequency=freq, presence=pres)
    want = x.float() - torch.tensor([0.0, 0.0, 0.75, math.inf])[:, None]
    assert same(got, want.to(dtype))
