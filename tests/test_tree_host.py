"""Refusals of the calls for drafted tokens (no device needed: arguments are
checked before anything is launched)."""
import ctypes
import math
import random

import pytest
import torch

from test_paged_host import ALIAS, ALIGN, FORMAT, NULL, OK, SHAPE, A, BAD_BATCH, BAD_CACHE, batch, cache


@pytest.fixture(scope="module")
def mt():
    import __graft_entry__
    __graft_entry__._libbuild().build()
    import quantized_gemv_epilogues_gb300 as m
    return m


def attention(mt, c=None, b=None, **kw):
    d = dict(q=A(5), q_stride=256, q_heads=4, visible=A(9), visible_ld=2, words=2, scale=0.1, window=0, sinks=0, out=A(6), out_stride=256,
             dtype=0, lse=A(7), ws=A(8), ws_bytes=1 << 30)
    d.update(kw)
    c, b = c or cache(mt), b or batch(mt)
    return mt.raw("mt_tree_attention")(d["q"], d["q_stride"], d["q_heads"], ctypes.byref(c), ctypes.byref(b), d["visible"], d["visible_ld"],
                                       d["words"], d["scale"], d["window"], d["sinks"], d["out"], d["out_stride"], d["dtype"], d["lse"],
                                       d["ws"], d["ws_bytes"], None)


def layout(mt, **kw):
    d = dict(parent=A(0), q_start=A(1), kv_len=A(2), B=3, T=50, positions=A(3), visible=A(4), visible_ld=2, words=2)
    d.update(kw)
    return mt.raw("mt_tree_layout")(*d.values(), None)


def probs(mt, **kw):
    d = dict(logits=A(0), ld=1000, dtype=1, R=4, V=1000, temperature=A(1), probs=A(2), probs_ld=1000)
    d.update(kw)
    return mt.raw("mt_token_probs")(*d.values(), None)


def verify(mt, **kw):
    d = dict(target=A(0), target_ld=1000, draft=A(1), draft_ld=1000, V=1000, tokens=A(2), parent=A(3), random=A(4), q_start=A(5), B=3, T=20,
             out_tokens=A(6), out_path=A(7), out_count=A(8), cols=5)
    d.update(kw)
    return mt.raw("mt_tree_verify")(*d.values(), None)


def keep(mt, caches=None, b=None, **kw):
    d = dict(path=A(5), count=A(6), cols=4, new_len=A(7))
    d.update(kw)
    caches = caches if caches is not None else [cache(mt), cache(mt, k=A(10), v=A(11))]
    arr = (ctypes.c_void_p * max(1, 2 * len(caches)))(*[p for c in caches for p in (c.k, c.v)])
    shape = caches[0] if caches else cache(mt)
    return mt.raw("mt_cache_keep")(ctypes.byref(shape), arr if caches else None, kw.get("L", len(caches)), ctypes.byref(b or batch(mt)),
                                   d["path"], d["count"], d["cols"], d["new_len"], None)


def test_cache_and_batch_refusals(mt):
    for kw, want in BAD_CACHE:
        assert attention(mt, c=cache(mt, **kw)) == want, kw
        assert keep(mt, [cache(mt, **kw)]) == want, kw
    for kw, want in BAD_BATCH:
        assert attention(mt, b=batch(mt, **kw)) == want, kw
        assert keep(mt, b=batch(mt, **kw)) == want, kw
    assert attention(mt, b=batch(mt, T=0)) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL), (dict(visible=None), NULL), (dict(dtype=2), FORMAT),
    (dict(q_heads=5), SHAPE), (dict(scale=math.nan), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(words=0), SHAPE),
    (dict(words=33, visible_ld=33), SHAPE), (dict(visible_ld=1), SHAPE), (dict(visible=A(9) + 2), ALIGN), (dict(ws_bytes=100), SHAPE),
    (dict(out=A(9)), ALIAS), (dict(lse=A(9)), ALIAS), (dict(ws=A(9)), ALIAS), (dict(out=A(5)), ALIAS)], ids=str)
def test_attention_refusals(mt, kw, want):
    assert attention(mt, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(parent=None), NULL), (dict(q_start=None), NULL), (dict(positions=None, visible=None), NULL), (dict(B=0), SHAPE),
    (dict(B=1025), SHAPE), (dict(T=-1), SHAPE), (dict(T=(1 << 22) + 1), SHAPE), (dict(words=0), SHAPE), (dict(words=33, visible_ld=40), SHAPE),
    (dict(visible_ld=1), SHAPE), (dict(parent=A(0) + 2), ALIGN), (dict(positions=A(3) + 1), ALIGN), (dict(visible=A(4) + 2), ALIGN),
    (dict(positions=A(0)), ALIAS), (dict(visible=A(1)), ALIAS), (dict(positions=A(2)), ALIAS), (dict(positions=A(4) + 16), ALIAS)], ids=str)
def test_layout_refusals(mt, kw, want):
    assert layout(mt, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), NULL), (dict(probs=None), NULL), (dict(dtype=2), FORMAT), (dict(R=-1), SHAPE), (dict(R=(1 << 22) + 1), SHAPE),
    (dict(V=0), SHAPE), (dict(V=(1 << 24) + 1, ld=1 << 25, probs_ld=1 << 25), SHAPE), (dict(ld=999), SHAPE), (dict(probs_ld=999), SHAPE),
    (dict(logits=A(0) + 2), ALIGN), (dict(probs=A(2) + 2), ALIGN), (dict(temperature=A(1) + 1), ALIGN), (dict(probs=A(0) + 400), ALIAS),
    (dict(probs=A(0), probs_ld=2000), ALIAS), (dict(probs=A(0), dtype=0), ALIAS), (dict(probs=A(1)), ALIAS)], ids=str)
def test_probs_refusals(mt, kw, want):
    assert probs(mt, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(target=None), NULL), (dict(tokens=None), NULL), (dict(parent=None), NULL), (dict(random=None), NULL), (dict(q_start=None), NULL),
    (dict(out_tokens=None), NULL), (dict(out_path=None), NULL), (dict(out_count=None), NULL), (dict(V=0), SHAPE), (dict(B=0), SHAPE),
    (dict(B=1025), SHAPE), (dict(T=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=(1 << 20) + 1), SHAPE), (dict(target_ld=999), SHAPE),
    (dict(draft_ld=999), SHAPE), (dict(target=A(0) + 2), ALIGN), (dict(random=A(4) + 1), ALIGN), (dict(out_path=A(7) + 2), ALIGN),
    (dict(out_tokens=A(0)), ALIAS), (dict(out_path=A(1) + 40), ALIAS), (dict(out_count=A(2)), ALIAS), (dict(out_path=A(6) + 8), ALIAS),
    (dict(out_count=A(5)), ALIAS)], ids=str)
def test_verify_refusals(mt, kw, want):
    assert verify(mt, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(path=None), NULL), (dict(count=None), NULL), (dict(caches=[]), NULL), (dict(L=0), SHAPE), (dict(L=1025), SHAPE),
    (dict(cols=0), SHAPE), (dict(cols=(1 << 20) + 1), SHAPE), (dict(path=A(5) + 2), ALIGN), (dict(new_len=A(7) + 1), ALIGN),
    (dict(new_len=A(3)), ALIAS), (dict(new_len=A(5)), ALIAS), (dict(new_len=A(10)), ALIAS), (dict(path=A(1)), ALIAS), (dict(count=A(11)), ALIAS)],
    ids=str)
def test_keep_refusals(mt, kw, want):
    assert keep(mt, **kw) == want


def test_caches_that_share_elements(mt):
    two = cache(mt, k=A(10), v=A(11))
    assert keep(mt, [cache(mt), two, cache(mt, k=None, v=A(12))]) == NULL
    assert keep(mt, [cache(mt), cache(mt, k=A(10), v=A(11) + 8)]) == ALIGN
    assert keep(mt, [cache(mt), two, cache(mt, k=A(12), v=A(10))]) == ALIAS        # a layer's values are another's keys
    assert keep(mt, [cache(mt), two, two]) == ALIAS
    assert keep(mt, [cache(mt), cache(mt, k=A(10), v=A(1) + 16)]) == ALIAS
    assert keep(mt, [cache(mt, v=A(0))]) == ALIAS
    # rows that share elements
    assert keep(mt, [cache(mt, token_stride=64, head_stride=64)]) == SHAPE


def test_layers_side_by_side_in_one_allocation(mt):
    # [page][layer][K, V][token][head][dim]: each cache spans the others, none shares a row.  (The calls end
    # at the checks that come after those of the caches: nothing is launched on made-up addresses.)
    row = 16 * 2 * 64
    L = 5

    def at(layer, side, shift=0):
        return A(0) + 2 * (row * (2 * layer + side) + shift)
    caches = [cache(mt, k=at(i, 0), v=at(i, 1), page_stride=2 * L * row) for i in range(L)]
    if not torch.cuda.is_available():
        assert keep(mt, caches) == mt.MT_ERR_CUDA
    caches[3] = cache(mt, k=at(3, 0), v=at(3, 1, -8), page_stride=2 * L * row)
    assert keep(mt, caches) == ALIAS


def test_layers_anywhere_against_their_elements(mt):
    # small caches at places and with strides of all kinds: an alias where, and only where, two share an element
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(1500):
        pages, page, heads, dim, L = rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 3), 16, rng.randint(1, 3)
        dims = [["pages", pages], ["page", page], ["heads", heads], ["layers", L], ["sides", 2]]
        rng.shuffle(dims)
        stride, step = {}, dim
        for name, n in dims:
            stride[name] = step
            step *= n
            if rng.random() < 0.2:
                step += 8 * rng.randint(1, 3)
        at = [stride["layers"] * i + stride["sides"] * j for i in range(L) for j in range(2)]
        if rng.random() < 0.5:
            at[rng.randrange(2 * L)] += 8 * rng.randint(0, 2 * step // 8)
        rows = [p * stride["pages"] + t * stride["page"] + h * stride["heads"] for p in range(pages) for t in range(page) for h in range(heads)]
        taken = [x + r + d for x in at for r in rows for d in range(0, dim, 8)]
        share = len(set(taken)) < len(taken)
        seen[share] += 1
        kw = dict(num_pages=pages, page_size=page, kv_heads=heads, head_dim=dim, page_stride=stride["pages"], token_stride=stride["page"],
                  head_stride=stride["heads"])
        caches = [cache(mt, k=A(0) + 2 * at[2 * i], v=A(0) + 2 * at[2 * i + 1], **kw) for i in range(L)]
        if share or not torch.cuda.is_available():  # (nothing is launched on made-up addresses)
            assert keep(mt, caches) == (ALIAS if share else mt.MT_ERR_CUDA), (dims, stride, at)
    assert min(seen.values()) > 100


def test_nothing_to_do(mt):
    assert layout(mt, T=0) == OK and layout(mt, T=0, parent=None, positions=None, visible=None) == OK
    assert probs(mt, R=0) == OK and probs(mt, R=0, logits=None, probs=None) == OK
    assert attention(mt, b=batch(mt, T=0), q=None, out=None, ws=None, lse=None, visible=None) == OK


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def calls(mt):
    """Each call with host tensors by name."""
    bf = torch.bfloat16
    paged = dict(k_cache=torch.zeros(4, 16, 2, 64, dtype=bf), v_cache=torch.zeros(4, 16, 2, 64, dtype=bf), pages=i32(2, 1).view(1, 2),
                 q_start=i32(0, 3), kv_len=i32(20))
    ws = torch.zeros(mt.mt_paged_attention_workspace_bytes(3, 1, 4, 2, 64), dtype=torch.uint8)
    return {
        "mt_tree_attention": dict(q=torch.zeros(3, 4, 64, dtype=bf), visible=i32(1, 3, 7).view(3, 1), max_q=3, scale=0.1,
                                  out=torch.zeros(3, 4, 64, dtype=bf), workspace=ws, lse=torch.zeros(3, 4), **paged),
        "mt_tree_layout": dict(parent=i32(-1, 0, 0), q_start=i32(0, 3), kv_len=i32(20), positions=i32(0, 0, 0), visible=i32(0, 0, 0).view(3, 1)),
        "mt_token_probs": dict(logits=torch.zeros(2, 50), probs=torch.zeros(2, 50), temperature=torch.ones(2)),
        "mt_tree_verify": dict(target=torch.zeros(3, 50), draft=torch.zeros(3, 50), tokens=i32(1, 2, 3), parent=i32(-1, 0, 0), random=torch.zeros(3),
                               q_start=i32(0, 3), out_tokens=i32(0, 0).view(1, 2), out_path=i32(0, 0).view(1, 2), out_count=i32(0)),
        "mt_cache_keep": dict(caches=[(paged["k_cache"], paged["v_cache"])], pages=paged["pages"], q_start=paged["q_start"],
                              kv_len=paged["kv_len"], path=i32(0, 2).view(1, 2), count=i32(2), new_len=i32(0)),
    }


BAD = [("mt_tree_attention", dict(visible=i32(1, 3).view(2, 1)), ValueError), ("mt_tree_attention", dict(visible=i32(1, 3, 7)), TypeError),
       ("mt_tree_attention", dict(visible=torch.zeros(3, 1)), TypeError), ("mt_tree_attention", dict(visible=None), TypeError),
       ("mt_tree_attention", dict(visible=torch.zeros(2, 3, dtype=torch.int32).t()), ValueError),
       ("mt_tree_attention", dict(kv_len=i32(1, 2)), ValueError),
       ("mt_tree_layout", dict(parent=torch.zeros(3)), TypeError), ("mt_tree_layout", dict(positions=i32(0, 0)), ValueError),
       ("mt_tree_layout", dict(kv_len=i32(0, 0)), ValueError), ("mt_tree_layout", dict(visible=i32(0, 0).view(2, 1)), ValueError),
       ("mt_tree_layout", dict(q_start=i32(0)), ValueError),
       ("mt_token_probs", dict(probs=torch.zeros(2, 49)), ValueError), ("mt_token_probs", dict(logits=torch.zeros(2, 50, dtype=torch.float16)), TypeError),
       ("mt_token_probs", dict(temperature=torch.ones(3)), ValueError), ("mt_token_probs", dict(probs=torch.zeros(50, 2).t()), ValueError),
       ("mt_tree_verify", dict(draft=torch.zeros(2, 50)), ValueError), ("mt_tree_verify", dict(tokens=i32(1, 2)), ValueError),
       ("mt_tree_verify", dict(random=torch.zeros(3, dtype=torch.float64)), TypeError), ("mt_tree_verify", dict(out_path=i32(0, 0, 0).view(1, 3)), ValueError),
       ("mt_tree_verify", dict(q_start=i32(0, 1, 3)), ValueError), ("mt_tree_verify", dict(target=torch.zeros(3, 50, dtype=torch.bfloat16)), TypeError),
       ("mt_cache_keep", dict(caches=[]), ValueError), ("mt_cache_keep", dict(path=i32(0, 2)), TypeError), ("mt_cache_keep", dict(count=i32(1, 2)), ValueError),
       ("mt_cache_keep", dict(new_len=torch.zeros(1)), TypeError),
       ("mt_cache_keep", dict(caches=[(torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16),)]), ValueError),
       ("mt_cache_keep", dict(caches=torch.zeros(3, 2, 4, 16, 2, 64)), TypeError),
       ("mt_cache_keep", dict(caches=torch.zeros(3, 3, 4, 16, 2, 64, dtype=torch.bfloat16)), ValueError),
       ("mt_cache_keep", dict(caches=torch.zeros(0, 2, 4, 16, 2, 64, dtype=torch.bfloat16)), ValueError),
       ("mt_cache_keep", dict(caches=torch.zeros(2, 4, 16, 2, 64, dtype=torch.bfloat16)), TypeError),
       ("mt_cache_keep", dict(caches=[(torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16),) * 2, (torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16),) * 2]), ValueError)]


@pytest.mark.parametrize("call,kw,err", BAD, ids=lambda x: x if isinstance(x, str) else ",".join(x) if isinstance(x, dict) else x.__name__)
def test_python_refusals(mt, call, kw, err):
    with pytest.raises(err):
        getattr(mt, call)(**{**calls(mt)[call], **kw}, stream=0)


CALLS = ["mt_tree_attention", "mt_tree_layout", "mt_token_probs", "mt_tree_verify", "mt_cache_keep"]


def test_host_caches_in_one_tensor(mt):
    kw = calls(mt)["mt_cache_keep"]
    with pytest.raises(mt.MTError, match="in host memory"):
        mt.mt_cache_keep(**{**kw, "caches": torch.zeros(3, 2, 4, 16, 2, 64, dtype=torch.bfloat16)}, stream=0)


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors(mt, call):
    with pytest.raises(mt.MTError, match="in host memory") as e:
        getattr(mt, call)(**calls(mt)[call], stream=0)
    assert e.value.status == NULL


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
def test_each_host_tensor_is_named(mt, call):
    good = {n: t.cuda() if torch.is_tensor(t) else t for n, t in calls(mt)[call].items()}
    if "caches" in good:
        good["caches"] = [tuple(x.cuda() for x in pair) for pair in good["caches"]]
    for name, t in good.items():
        if torch.is_tensor(t):
            with pytest.raises(mt.MTError, match=f"^{call}: {name}: "):
                getattr(mt, call)(**{**good, name: t.cpu()})
    getattr(mt, call)(**good)
    torch.cuda.synchronize()
