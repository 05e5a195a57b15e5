"""mt_token_probs for many rows and for vocabularies that no cluster's registers
hold, which another kernel takes: the cases of test_gpu_token_probs.py there."""
import math

import pytest
import torch

from test_gpu_token_probs import DTYPES, check, logits, mt  # noqa: F401

pytestmark = pytest.mark.gpu


@DTYPES
@pytest.mark.parametrize("R,V", [(310, 21001), (700, 24576), (350, 32003), (20, 170001), (3, 500003)])
def test_sizes(mt, dtype, R, V):  # noqa: F811
    check(mt, logits(R, V, dtype, V), [[1.0, 0.0, 0.6, math.inf, 0.02][r % 5] for r in range(R)])


@DTYPES
@pytest.mark.parametrize("pad,out_pad", [(1, 0), (0, 1), (3, 3), (8, 4), (5, 2)])
def test_strides(mt, dtype, pad, out_pad):  # noqa: F811
    check(mt, logits(320, 21011, dtype, 5), [0.7] * 320, pad, out_pad)
    check(mt, logits(320, 21011, dtype, 5), [0.0] * 320, pad, out_pad)


@DTYPES
@pytest.mark.parametrize("V", [21013, 330007])
def test_masks_nan_and_infinities(mt, dtype, V):  # noqa: F811
    lowest, highest = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = logits(20, V, dtype, 3)
    x[0] = -math.inf
    x[1] = -math.inf
    x[1, V - 1] = -5.0
    x[2, V // 2] = math.nan
    x[3, 0] = math.inf
    x[4, ::3] = -math.inf
    x[5] = 1.5
    x[6, V - 1] = math.nan
    x[7] = lowest
    x[8] = lowest
    x[8, 3] = highest
    x[9, 1] = math.nan
    x[10, :V - 1] = -math.inf
    x[10, V - 1] = math.nan
    x[11, 5], x[11, 7] = math.inf, -math.inf
    x[12, V - 1] = math.inf
    x[13] = -math.inf
    x[13, V // 2 - 40:V // 2 + 40] = torch.linspace(-3, 3, 80).to(dtype)
    x[14] = highest
    x[15] += 300.0
    x[16] -= 1000.0
    x[17] += 20000.0
    x[18] *= 1e30
    x[19] *= 1e-30
    many = 1 if V > 100000 else 17  # rows enough for the kernel
    for t in ([1.0] * 20, [0.0] * 20, [math.inf] * 20, [0.03] * 20, [1e4] * 20, [1e-20] * 20):
        check(mt, x.repeat(many, 1), t * many)


@DTYPES
def test_the_first_of_equal_logits(mt, dtype):  # noqa: F811
    for pad in (0, 3):
        x = logits(320, 21013, dtype, 7).clamp(max=2.0)
        check(mt, x, [0.0] * 320, pad)
        x[::2, 21011:] = 9.0                       # behind the last vector
        x[1::2, :3] = 9.0                          # and before the first, where rows start between boundaries
        x[::3, 10000] = 9.0
        check(mt, x, [0.0] * 320, pad)


@DTYPES
def test_logits_far_from_zero_in_registers(mt, dtype):  # noqa: F811
    x = logits(8, 5003, dtype, 9)
    for r, shift in enumerate((300.0, -300.0, 5000.0, -5000.0, 1e6, -1e6, 1e30, -1e30)):
        x[r] += shift
    for t in (1.0, 0.01, 50.0, 1e-25, 1e25):
        check(mt, x, [t] * 8)


def test_in_place(mt):  # noqa: F811
    check(mt, logits(330, 21013, torch.float32, 4), [0.4] * 330, pad=3, in_place=True)
    check(mt, logits(4, 400001, torch.float32, 4), [1.0, 0.0, 0.4, 2.0], pad=1, in_place=True)


@DTYPES
def test_without_programmatic_launch_and_equal_runs(mt, dtype):  # noqa: F811
    for R, V in ((330, 21013), (5, 60000), (9, 300)):
        x = logits(R, V, dtype, 11).cuda()
        a, b = torch.empty(R, V, device="cuda"), torch.empty(R, V, device="cuda")
        mt.mt_token_probs(x, a)
        mt.mt_set_option(mt.MT_OPT_PDL, 0)
        try:
            mt.mt_token_probs(x, b)
        finally:
            mt.mt_set_option(mt.MT_OPT_PDL, 1)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
