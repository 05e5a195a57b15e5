"""GPU tests of mt_rope_append's sines and cosines relative to their own size:
one element of each pair is zero, so that nothing else hides them."""
import math

import pytest
import torch

from test_gpu_rope_append import mt  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

# the rounding to bf16, and in fp32 the sine's and cosine's own error (a few
# units in the last place) and a product
REL = 2.0 ** -8 + 16 * 2.0 ** -24


@pytest.mark.parametrize("adjacent", [False, True], ids=["half", "adjacent"])
@pytest.mark.parametrize("tokens", [9, 2000, 9000])
def test_small_sines_and_cosines(mt, tokens, adjacent):  # noqa: F811
    D, half = 64, 32
    freq = torch.tensor([theta ** (-2 * i / 64) for theta in (1e4, 5e6, 1e9) for i in (0, 17, 30, 31)]
                        + [math.pi / 2, math.pi, 2 * math.pi, math.pi / 4, 3.0, 1e-11, -1e-7, 0.0], dtype=torch.float64)
    freq = freq.repeat(2)[:half].float()
    pos = torch.arange(tokens) - 4
    pos[5:] = torch.where(pos[5:] % 3 == 0, pos[5:] * 1009, pos[5:])
    x = torch.zeros(tokens, 2, D)
    first = (torch.arange(D) % 2 == 0) if adjacent else (torch.arange(D) < half)
    x[:, 0, first] = 1.5   # its partner gets the sine, itself the cosine
    x[:, 1, ~first] = 1.5
    x = x.to(torch.bfloat16).cuda()
    out = torch.empty_like(x)
    cache = torch.zeros(2, -(-tokens // 16), 16, 2, D, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    mt.mt_rope_append(x, x, x, pos.to(torch.int32).cuda(), freq.cuda(), out, cache[0], cache[1],
                      torch.arange(cache.shape[1], **i32)[None], torch.tensor([0, tokens], **i32), torch.tensor([tokens], **i32),
                      pairing=mt.MT_ROPE_ADJACENT if adjacent else mt.MT_ROPE_HALF)
    got = out.cpu().double()
    angle = pos[:, None].double() * freq.double()
    want = torch.zeros(tokens, 2, D, dtype=torch.float64)
    want[:, 0, first], want[:, 0, ~first] = 1.5 * angle.cos(), 1.5 * angle.sin()
    want[:, 1, first], want[:, 1, ~first] = -1.5 * angle.sin(), 1.5 * angle.cos()
    # the reference's own product is rounded to 2^-53 of the angle, and the kernel's
    # fraction of a turn to 2^-64 a position
    slack = 1.5 * (angle.abs() * 2.0 ** -53 + 2 * math.pi * 2.0 ** -64 * pos.abs()[:, None].double())
    slack = torch.cat([slack, slack], 1) if not adjacent else slack.repeat_interleave(2, 1)
    assert bool(((got - want).abs() <= REL * want.abs() + slack[:, None] + 2.0 ** -133).all())
