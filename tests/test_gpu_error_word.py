"""The device error word keeps a timeout that a later call's bad page follows
(the wait runs out on its own: arrivals that nothing makes, no GPU fault)."""
import numpy as np
import pytest
import torch

import synth
from gpu_layers import DevLayer, plan_layer
from paged_util import Paged
from parity_util import dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    m.mt_device_error(True)
    yield m
    assert m.mt_device_error(True) == 0


def expire_a_wait(mt):
    wl = synth.TINY.with_(layers=2)
    layers = [plan_layer(DevLayer(mt, wl, l)) for l in range(2)]
    vals = dev_bf16(np.stack([synth.host_bf16(wl.d, synth.seed_for(wl.wid, l, synth.T_VALUES), synth.ACT) for l in range(2)]))
    r0 = dev_bf16(synth.host_bf16(wl.d, synth.seed_for(wl.wid, 0, synth.T_RESIDUAL), synth.ACT))
    plan = mt.mt_mlp_plan_create(layers, wl.d, wl.f, wl.group, wl.fmt, wl.eps)
    mt.mt_set_option(mt.MT_OPT_TEST_BARRIER_EXTRA, 1)
    try:
        mt.mt_mlp_plan_run(plan, vals, r0, torch.empty(wl.d, dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
    finally:
        mt.mt_set_option(mt.MT_OPT_TEST_BARRIER_EXTRA, 0)
        mt.mt_mlp_plan_destroy(plan)


def bad_page(mt, call, page):
    p = Paged([(3, 40)], 4, 2, 64, page=page, seed=1)
    p.pages[0, 2] = p.num_pages
    q, k, v, pages, q_start, kv_len = p.cuda()
    out = torch.empty_like(q)
    if call == "attention":
        ws = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, 1, 4, 2, 64), dtype=torch.uint8, device="cuda")
        mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, 3, 0.125, out, ws)
    else:
        new = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        mt.mt_rope_append(q, new, new, torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda"), out, k, v,
                          pages, q_start, kv_len)
    torch.cuda.synchronize()


@pytest.mark.parametrize("call,page", [("attention", 16), ("attention", 12), ("rope", 16)])
def test_a_bad_page_does_not_replace_a_timeout(mt, call, page):
    expire_a_wait(mt)
    assert mt.mt_device_error(False) == mt.MT_ERR_TIMEOUT
    bad_page(mt, call, page)
    assert mt.mt_device_error(True) == mt.MT_ERR_TIMEOUT
    bad_page(mt, call, page)
    assert mt.mt_device_error(True) == mt.MT_ERR_PAGE
