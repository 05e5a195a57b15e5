"""GPU test of a batch of trees and of a prompt longer than the bits of a row:
one call for each, on the same rows."""
import math

import pytest
import torch

from paged_util import Paged, attention_bounds, attention_ref, check
from tree_util import bit_rows, mixed_tree, seen_of, tree_attention_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    m.mt_device_error(True)
    yield m
    assert m.mt_device_error(True) == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 3)])
@pytest.mark.parametrize("page", [16, 12], ids=["chunk-kernel", "rows-kernel"])
def test_trees_and_a_long_prompt(mt, page, window, sinks):
    p = Paged([(25, 403), (7, 7), (60, 95), (1100, 1300), (30, 50)], 4, 2, 64, page=page, seed=2)
    trees = 3  # the first of them; then a prompt of 1100 tokens and one of 30
    seen = [seen_of(mixed_tree(n, b)) for b, (n, _) in enumerate(p.lens[:trees])]
    visible = bit_rows(seen, int(p.q_start[trees]), 2)
    q, k, v, pages, q_start, kv_len = p.cuda()
    out = torch.full((p.T, p.hq, p.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.T, p.hq), 7.0, device="cuda")
    space = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, len(p.lens), p.hq, p.hkv, p.d), dtype=torch.uint8, device="cuda")
    scale = 1 / math.sqrt(p.d)
    rows = int(p.q_start[trees])
    mt.mt_tree_attention(q[:rows], k, v, pages[:trees], q_start[:trees + 1], kv_len[:trees], visible.cuda(), 60, scale, out[:rows], space,
                         lse=lse[:rows], window=window, sinks=sinks)
    mt.mt_paged_attention(q, k, v, pages[trees:], q_start[trees:], kv_len[trees:], 1100, scale, out, space, lse=lse, window=window, sinks=sinks)
    torch.cuda.synchronize()
    # a prompt's token sees those of its window among the new ones, too
    chunk = [torch.ones(n, n, dtype=torch.bool).tril() for n, _ in p.lens[trees:]]
    ref = tree_attention_ref(p, seen + chunk, scale, window, sinks)
    if window:
        for r, x in zip(ref, attention_ref(p, scale, window, sinks)):
            r[rows:] = x[rows:]
    tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
    check(lse, ref[1], tol_lse, "lse")
    check(out, ref[0], tol_out, "out")
