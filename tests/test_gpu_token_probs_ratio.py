"""GPU tests of mt_token_probs' exponentials by themselves: every probability
over the row's largest, in which the sum and its rounding cancel."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    return m


# Relative to p / max p.  Both are off by an exponential (2^-22), its factor's two roundings and up to
# two in the scaling (2^-24 each; one row in registers: the warp's factor is another exponential
# with two roundings, and its product with 1 / sum one).  The argument's part is below
# 2^-30: 2^-40 of a product of 125, and the square of its rest (5.1e-5 at the most) in the factor.
# A rounding to fp32 of an argument of 40 to 125 alone would be up to 2^-18 or more.
ONE = 2.0 ** -22 + 4 * 2.0 ** -24
TOLERANCE = 2 * (ONE + 2.0 ** -22 + 4 * 2.0 ** -24) + 2.0 ** -30


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
# rows in registers and in two passes; blocks of a row
@pytest.mark.parametrize("R,V", [(3, 200), (3, 5000), (9, 151936), (5, 300007), (448, 4000), (448, 50257), (200, 40001)])
def test_small_probabilities(mt, dtype, R, V):
    g = torch.Generator().manual_seed(V)
    # the largest at 20, the others 0 to 85 below it, on a grid where differences are exact
    # (bf16 holds quarters up to 64)
    step = 4 if dtype is torch.bfloat16 else 1024
    x = 20 - torch.randint(0, 84 * step, (R, V), generator=g) / step
    x[:, V // 3] = 20
    assert torch.equal(x.to(dtype).float(), x)
    t = torch.tensor([[1.0, 0.99, 1.3, 2.0][r % 4] for r in range(R)])
    out = torch.empty(R, V, device="cuda")
    mt.mt_token_probs(x.to(dtype).cuda(), out, t.cuda())
    want = torch.exp((x.double() - 20) / t.double()[:, None])
    got = out.cpu().double()
    normal = want > 2.0 ** -125 * want.sum(1, keepdim=True)  # steps of 2^-149 are all that is left of smaller ones
    got = got / got[:, V // 3:V // 3 + 1]
    worst = float(((got - want).abs() / want)[normal].max())
    assert float(want[normal].min()) < 2.0 ** -100
    assert worst <= TOLERANCE, worst
