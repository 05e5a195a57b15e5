"""The Python calls around the projections refuse tensors in pageable host
memory, whose addresses mean nothing to a kernel; pinned ones are taken."""
import pytest
import torch


@pytest.fixture(scope="module")
def mt():
    import __graft_entry__
    __graft_entry__._libbuild().build()
    import quantized_gemv_epilogues_gb300 as m
    return m


def calls(mt, device):
    """Each call with its tensors by name."""
    bf, i32 = dict(dtype=torch.bfloat16, device=device), dict(dtype=torch.int32, device=device)
    g = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(device)

    cache = dict(k_cache=normal(4, 16, 2, 64).to(torch.bfloat16), v_cache=normal(4, 16, 2, 64).to(torch.bfloat16),
                 pages=torch.tensor([[2, 1]], **i32), q_start=torch.tensor([0, 3], **i32), kv_len=torch.tensor([20], **i32))
    q = normal(3, 4, 64).to(torch.bfloat16)
    f32 = dict(device=device)
    return {
        "mt_rope_append": dict(q=q, k=normal(3, 2, 64).to(torch.bfloat16), v=normal(3, 2, 64).to(torch.bfloat16),
                               positions=torch.arange(3, **i32), inv_freq=torch.ones(32, **f32), q_out=torch.zeros(3, 4, 64, **bf),
                               axis=torch.zeros(32, dtype=torch.uint8, device=device), q_norm=torch.ones(64, **bf),
                               k_norm=torch.ones(64, **bf), **cache),
        "mt_paged_attention": dict(q=q, max_q=3, scale=0.125, out=torch.zeros(3, 4, 64, **bf), lse=torch.zeros(3, 4, **f32),
                                   workspace=torch.zeros(mt.mt_paged_attention_workspace_bytes(3, 1, 4, 2, 64), dtype=torch.uint8,
                                                         device=device), **cache),
        "mt_logit_penalties": dict(logits=normal(1, 50), out=torch.zeros(1, 50, **f32), history=torch.tensor([3, 3, 7], **i32),
                                   history_start=torch.tensor([0, 3], **i32), prompt_len=torch.tensor([1], **i32),
                                   repetition=torch.full((1,), 1.5, **f32), presence=torch.ones(1, **f32),
                                   frequency=torch.ones(1, **f32), bias_ids=torch.tensor([4], **i32), bias_values=torch.ones(1, **f32),
                                   bias_start=torch.tensor([0, 1], **i32), allowed=torch.full((1, 2), -1, **i32)),
    }


@pytest.mark.parametrize("call", ["mt_rope_append", "mt_paged_attention", "mt_logit_penalties"])
def test_host_tensors(mt, call):
    with pytest.raises(mt.MTError, match="in host memory") as e:
        getattr(mt, call)(**calls(mt, "cpu")[call], stream=0)
    assert e.value.status == mt.MT_ERR_NULL


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["mt_rope_append", "mt_paged_attention", "mt_logit_penalties"])
def test_each_host_tensor_is_named_and_pinned_ones_are_taken(mt, call):
    good = calls(mt, "cuda")[call]
    for name, t in good.items():
        if torch.is_tensor(t):
            with pytest.raises(mt.MTError, match=f"^{call}: {name}: "):
                getattr(mt, call)(**{**good, name: t.cpu().view(t.shape)})
    outs = [n for n in ("q_out", "out", "lse", "k_cache", "v_cache") if n in good]
    getattr(mt, call)(**good)
    torch.cuda.synchronize()
    want = [good[n].clone() for n in outs]
    # a server's small arrays, read where the host wrote them
    again = calls(mt, "cuda")[call]
    for n in ("q_start", "kv_len", "positions", "history_start", "prompt_len", "repetition"):
        if n in again:
            again[n] = again[n].cpu().pin_memory()
    getattr(mt, call)(**again)
    torch.cuda.synchronize()
    assert all(torch.equal(again[n], w) for n, w in zip(outs, want))


def test_lists_without_their_starts_are_refused_as_before(mt):
    x, ids = torch.zeros(1, 50), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(history=ids), dict(bias_ids=ids, bias_values=torch.zeros(2))):
        with pytest.raises(mt.MTError) as e:
            mt.mt_logit_penalties(x, torch.zeros(1, 50), **kw, stream=0)
        assert e.value.status == mt.MT_ERR_NULL


def test_a_workspace_of_repeated_elements(mt):
    # nbytes counts an expanded tensor's one element as often as it is repeated
    kw = calls(mt, "cpu")["mt_paged_attention"]
    kw["workspace"] = torch.zeros(1, dtype=torch.uint8).expand(kw["workspace"].numel())
    with pytest.raises(ValueError, match="contiguous"):
        mt.mt_paged_attention(**kw, stream=0)
