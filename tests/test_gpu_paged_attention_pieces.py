"""GPU tests of the chunk kernel's ring of pieces: chunks that fill both of a
CTA's tiles, followed in the same CTA by many short pieces with rows in the
first tile only, which the second tile's warps have to keep pace with although
nothing of theirs is needed there."""
import pytest
import torch

from paged_util import Paged
from test_gpu_paged_attention import compare, mt  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(12, 4, 128), (8, 8, 64), (32, 8, 64)], ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("singles", [1, 4, 11])
def test_short_single_tokens_after_a_chunk(mt, heads, singles):  # noqa: F811
    # one CTA's stretch holds several chunks' ends and the one- and two-block
    # texts behind them; groups of 3 leave by the slowest of the row stores, and
    # the chunk's second tile has a block more than the first every other time
    full = 256 // (heads[0] // heads[1])
    lens = []
    while len(lens) < 300:
        lens.append((full - len(lens) % 5, full + 40 + len(lens) % 128))
        lens += [(1, 1 + (37 * (len(lens) + i)) % 256) for i in range(singles)]
    p = Paged(lens, *heads, page=16, seed=31)
    compare(mt, p)
    assert mt.mt_device_error(False) == 0


def test_single_pieces_of_several_blocks_after_a_chunk(mt):  # noqa: F811
    # growing scores: the first tile's rows are rescaled, block after block,
    # while the second tile's rows still leave
    lens = []
    while len(lens) < 240:
        lens += [(85, 130 + len(lens) % 60), (1, 390), (1, 5), (2, 260)]
    p = Paged(lens, 12, 4, 128, page=16, seed=32, q_scale=4.0)
    for b, (_, kv) in enumerate(lens):
        p.keys[b] *= torch.linspace(0.2, 2.0, kv)[:, None, None].to(torch.bfloat16)
        for i in range(-(-kv // 16)):
            n = min(16, kv - 16 * i)
            p.k[p.pages[b, i], :n] = p.keys[b][16 * i:16 * i + n]
    compare(mt, p)
    assert mt.mt_device_error(False) == 0
