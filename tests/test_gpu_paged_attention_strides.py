"""GPU tests of mt_paged_attention on caches whose dimensions of one entry have
strides that mean nothing."""
import pytest
import torch

from paged_util import Paged
from test_gpu_paged_attention import mt, run  # noqa: F401  (mt: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("stride", [0, 8, 24, 1 << 30])
@pytest.mark.parametrize("which", ["head", "page"])
def test_strides_of_dimensions_of_one_entry(mt, which, stride, d):  # noqa: F811
    page = 128 if which == "page" else 16
    p = Paged([(5, 77)], 4, 1, d, page=page, seed=27, spare=0 if which == "page" else 2)
    want, wl = run(mt, p, 0.1)
    q, k, v, pages, q_start, kv_len = p.cuda()
    st = list(k.stride())
    st[2 if which == "head" else 0] = stride
    k, v = k.as_strided(k.shape, st), v.as_strided(v.shape, st)
    out, lse = torch.empty_like(q), torch.empty(p.T, 4, device="cuda")
    ws = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, 1, 4, 1, d), dtype=torch.uint8, device="cuda")
    mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, 5, 0.1, out, ws, lse=lse)
    assert torch.equal(out, want) and torch.equal(lse, wl)
