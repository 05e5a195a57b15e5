"""Integers beyond 32 bits in the Python calls: taken for what they mean, or
refused, never cut to their lower bits."""
import pytest
import torch

from paged_util import Paged
from test_gpu_paged_attention import compare, mt  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks,as_window,as_sinks", [
    (2 ** 32 + 5, 0, 0, 0), (2 ** 31, 3, 0, 0), (2 ** 63 - 1, 0, 0, 0), (64, 2 ** 32, 64, 1000), (64, 2 ** 32 + 2, 64, 1000),
    (64, 2 ** 31, 64, 1000)])
@pytest.mark.parametrize("lens", [[(1, 500), (1, 3)], [(200, 333), (2, 9)]], ids=["decode", "chunk"])
def test_windows_and_sinks(mt, lens, window, sinks, as_window, as_sinks):  # noqa: F811
    p = Paged(lens, 8, 2, 64, page=16, seed=25)
    q, k, v, pages, q_start, kv_len = p.cuda()
    ws = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, len(lens), 8, 2, 64), dtype=torch.uint8, device="cuda")
    got, want = torch.empty_like(q), torch.empty_like(q)
    mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, p.max_q, 0.125, got, ws, window=window, sinks=sinks)
    mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, 2 ** 40, 0.125, want, ws, window=as_window, sinks=as_sinks)
    assert torch.equal(got, want)
    compare(mt, p, as_window, as_sinks)


@pytest.mark.parametrize("kw", [dict(window=-1), dict(window=-2 ** 32 + 5), dict(sinks=-2 ** 40 + 1), dict(window=-2 ** 32)], ids=str)
def test_negative_ones_are_refused(mt, kw):  # noqa: F811
    p = Paged([(1, 20)], 4, 2, 64, page=16, seed=26)
    q, k, v, pages, q_start, kv_len = p.cuda()
    ws = torch.empty(mt.mt_paged_attention_workspace_bytes(1, 1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    with pytest.raises(mt.MTError) as e:
        mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, 1, 0.125, torch.empty_like(q), ws, **kw)
    assert e.value.status == mt.MT_ERR_SHAPE


def test_a_history_of_2_to_the_31(mt):  # noqa: F811
    x = torch.zeros(1, 9, device="cuda")
    history = torch.empty(2 ** 31, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mt.mt_logit_penalties(x, torch.empty_like(x), history=history, history_start=start)
