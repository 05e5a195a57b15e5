"""GPU tests of mt_paged_attention with values and bounds that show the loss of
any one key's value, on texts that are split over the GPU too."""
import pytest
import torch

from attention_values import CASES, coded, reference
from paged_util import check
from test_gpu_paged_attention import mt, run  # noqa: F401  (mt: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_every_key_counts_once(mt, name, dtype):  # noqa: F811
    lens, heads, page, window, sinks = CASES[name]
    scale = heads[2] ** -0.5
    p = coded(lens, *heads, page=page, seed=50)
    out, _ = run(mt, p, scale, window, sinks, dtype)
    # fp32 outputs, pages of 12 and head size 256 take the kernel with weights of two bf16
    one = dtype == torch.bfloat16 and page % 8 == 0 and heads[2] <= 128
    want, tol, _ = reference(p, scale, window, sinks, 2.0 ** -8 if one else 2.0 ** -16, dtype)
    check(out, want, tol, "out")
