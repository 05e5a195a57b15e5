"""GPU tests of mt_paged_attention against a 64-bit reference: head layouts,
page sizes, lengths from zero on, windows and sinks, cache orders, strides,
stale NaN slots, page-table entries that must not be followed."""
import math

import pytest
import torch

from paged_util import Paged, attention_bounds, attention_ref, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    m.mt_device_error(True)
    yield m
    assert m.mt_device_error(True) == 0


def run(mt, p, scale, window=0, sinks=0, dtype=torch.bfloat16, max_q=None, out_pad=0, stream=None):
    q, k, v, pages, q_start, kv_len = p.cuda()
    out = torch.full((p.T, p.hq * p.d + out_pad), 7.0, dtype=dtype, device="cuda")
    view = out[:, :p.hq * p.d].unflatten(1, (p.hq, p.d))
    lse = torch.full((p.T, p.hq), 7.0, dtype=torch.float32, device="cuda")
    # a workspace of NaN: its contents are of no account
    ws = torch.full((mt.mt_paged_attention_workspace_bytes(p.T, len(p.lens), p.hq, p.hkv, p.d) // 4,), math.nan, device="cuda")
    torch.cuda.synchronize()
    mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, p.max_q if max_q is None else max_q, scale, view, ws, lse=lse,
                          window=window, sinks=sinks, stream=stream)
    torch.cuda.synchronize()
    rows = int(p.q_start[-1])
    assert bool((out[rows:] == 7).all()) and bool((out[:, p.hq * p.d:] == 7).all()), "rows of no sequence were written"
    return view[:rows], lse[:rows]


def compare(mt, p, window=0, sinks=0, dtype=torch.bfloat16, rounding=2.0 ** -8, **kw):
    scale = 1.0 / math.sqrt(p.d)
    out, lse = run(mt, p, scale, window, sinks, dtype, **kw)
    ref = attention_ref(p, scale, window, sinks)
    tol_out, tol_lse = attention_bounds(p, ref, rounding if dtype == torch.bfloat16 else 2.0 ** -16, dtype)
    check(lse, ref[1], tol_lse, "lse")
    check(out, ref[0], tol_out, "out")


HEADS = [(4, 4, 64), (8, 2, 128), (14, 2, 64), (3, 1, 96), (6, 2, 72), (16, 1, 128), (2, 2, 16), (5, 5, 128), (8, 1, 256), (40, 8, 40)]


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 777)], [(1, 64), (1, 65), (1, 1), (1, 300)]], ids=["one", "777", "ragged"])
def test_single_tokens(mt, heads, lens):
    compare(mt, Paged(lens, *heads, page=16, seed=1))


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("lens", [[(5, 70), (17, 17), (1, 200), (33, 129)], [(150, 400), (3, 3)], [(300, 300)]],
                         ids=["short", "chunk", "prompt"])
def test_chunks(mt, heads, lens):
    compare(mt, Paged(lens, *heads, page=16, seed=2))


@pytest.mark.parametrize("heads", [(128, 1, 64), (100, 1, 64), (33, 1, 128), (66, 2, 88), (7, 7, 120), (32, 1, 64), (4, 4, 104)],
                         ids=lambda h: "x".join(map(str, h)))
def test_other_groups_and_head_sizes(mt, heads):
    compare(mt, Paged([(1, 300), (5, 70), (41, 200), (3, 3)], *heads, page=16, seed=20))
    compare(mt, Paged([(1, 300), (41, 200)], *heads, page=16, seed=20), window=50, sinks=2)


@pytest.mark.parametrize("page", [1, 3, 8, 20, 24, 48, 64, 128, 256])
@pytest.mark.parametrize("lens", [[(1, 130), (1, 401)], [(140, 333), (2, 9)]], ids=["decode", "chunk"])
def test_page_sizes(mt, page, lens):
    compare(mt, Paged(lens, 8, 2, 64, page=page, seed=3))


@pytest.mark.parametrize("order", ["hnd", "kv"])
@pytest.mark.parametrize("lens", [[(1, 130), (1, 401)], [(140, 333), (2, 9)]], ids=["decode", "chunk"])
def test_cache_orders_and_row_strides(mt, order, lens):
    compare(mt, Paged(lens, 8, 2, 128, page=16, order=order, seed=4, q_pad=24, rows_pad=3), out_pad=40)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (64, 4), (100, 70), (1000, 3), (129, 0), (7, 1000)])
@pytest.mark.parametrize("lens", [[(1, 500), (1, 3), (1, 128)], [(200, 333), (2, 9), (1, 600)]], ids=["decode", "chunk"])
def test_window_and_sinks(mt, window, sinks, lens):
    for heads in ((8, 2, 128), (7, 1, 64)):
        compare(mt, Paged(lens, *heads, page=16, seed=5), window, sinks)


@pytest.mark.parametrize("window", [512, 513, 2 ** 30, 2 ** 31 - 100, 2 ** 31 - 1])
@pytest.mark.parametrize("lens", [[(1, 500), (1, 3)], [(200, 512), (9, 4), (1, 300)]], ids=["decode", "chunk"])
def test_windows_wider_than_any_text(mt, window, lens):
    # (9, 4): the first tokens' positions are negative; pages of 12 are not the chunk kernel's
    for page in (16, 12):
        for sinks in (0, 2 ** 31 - 1):
            compare(mt, Paged(lens, 8, 2, 64, page=page, seed=24), window, sinks)


@pytest.mark.parametrize("max_q", [1, 1000])
def test_the_hint_changes_no_result(mt, max_q):
    compare(mt, Paged([(1, 130), (90, 401), (1, 1)], 8, 2, 64, page=16, seed=6), max_q=max_q)


def test_sequences_without_tokens_and_rows_that_see_nothing(mt):
    # no new tokens; an empty cache; more new tokens than the cache has room for
    for lens in ([(0, 40), (1, 0), (6, 4), (0, 0), (1, 33), (0, 5)], [(200, 150), (0, 9), (130, 0)]):
        compare(mt, Paged(lens, 8, 2, 64, page=16, seed=7))


def test_all_sequences_empty(mt):
    p = Paged([(0, 40), (0, 0)], 4, 2, 64, page=16, seed=8, rows_pad=2)
    out, lse = run(mt, p, 0.1)
    assert out.numel() == 0


@pytest.mark.parametrize("lens", [[(1, 300), (1, 40)], [(150, 300)]], ids=["decode", "chunk"])
def test_fp32_output(mt, lens):
    for heads in ((8, 2, 128), (14, 2, 64), (8, 1, 256)):
        compare(mt, Paged(lens, *heads, page=16, seed=9), dtype=torch.float32)


def test_weights_of_the_rows_kernel_are_rounded_to_two_bf16(mt):
    # pages of 12 tokens are not the chunk kernel's
    compare(mt, Paged([(1, 900), (2, 300)], 8, 2, 128, page=12, seed=10), rounding=2.0 ** -16)


def test_large_scores(mt):
    # one weight takes nearly all: the maximum moves late, the sum stays near 1
    compare(mt, Paged([(1, 700), (140, 300)], 8, 2, 64, page=16, seed=11, q_scale=30.0))
    compare(mt, Paged([(1, 700), (3, 300)], 8, 2, 64, page=16, seed=11, q_scale=30.0))


def test_pages_that_no_token_sees_are_not_followed(mt):
    # entries between the sinks and the window are -1 (given back): no error, no change
    for lens, window in (([(1, 900)], 100), ([(140, 900)], 100)):
        p = Paged(lens, 8, 2, 64, page=16, seed=12)
        first = (lens[0][1] - lens[0][0] - window + 1) // 16
        p.pages[0, 1:first] = -1
        compare(mt, p, window, 5)
        assert mt.mt_device_error(False) == 0


@pytest.mark.parametrize("page", [16, 64, 128, 12])
@pytest.mark.parametrize("window,sinks", [(37, 0), (100, 5), (130, 131), (1, 20)])
def test_keys_that_a_token_does_not_see_may_be_nan(mt, page, window, sinks):
    # one new token each: every key outside its window and sinks holds NaN and infinities
    p = Paged([(1, 500), (1, 129), (1, 40), (1, 257)], 8, 2, 64, page=page, seed=23)
    for b, (_, kv) in enumerate(p.lens):
        for j in range(sinks, kv - window):
            for x, bad in ((p.k, math.nan), (p.v, math.nan if j % 2 else math.inf)):
                x[p.pages[b, j // page], j % page] = bad
    compare(mt, p, window, sinks)


@pytest.mark.parametrize("page", [16, 128])
def test_tokens_after_a_tile_may_be_nan(mt, page):
    # one head to a group: a tile is 256 tokens, and the last token of 300 is NaN
    p = Paged([(300, 300)], 2, 2, 64, page=page, seed=24)
    p.k[p.pages[0, 299 // page], 299 % page] = math.nan
    p.v[p.pages[0, 299 // page], 299 % page] = math.nan
    p.k[p.pages[0, 257 // page], 257 % page] = math.nan
    p.v[p.pages[0, 257 // page], 257 % page] = math.inf
    out, lse = run(mt, p, 0.125)
    ref = attention_ref(p, 0.125)
    tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
    check(out[:256], ref[0][:256], tol_out[:256])
    check(lse[:256], ref[1][:256], tol_lse[:256])


@pytest.mark.parametrize("lens", [[(1, 100)], [(130, 200)]], ids=["decode", "chunk"])
def test_page_out_of_range_is_reported(mt, lens):
    # the entry is checked on the device before it is followed; its keys count as zeros
    p = Paged(lens, 4, 2, 64, page=16, seed=13)
    bad = p.pages.clone()
    bad[0, 2] = p.num_pages
    p.keys[0][32:48] = 0
    p.values[0][32:48] = 0
    p.pages = bad
    scale = 0.125
    out, lse = run(mt, p, scale)
    assert mt.mt_device_error(True) == mt.MT_ERR_PAGE
    ref = attention_ref(p, scale)
    tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
    check(out, ref[0], tol_out)
    check(lse, ref[1], tol_lse)


@pytest.mark.parametrize("lens", [[(1, 5000)] * 3, [(70, 3000), (1, 4000)], [(400, 2500)]], ids=["decode", "mixed", "chunk"])
def test_two_calls_give_the_same_bits(mt, lens):
    p = Paged(lens, 8, 2, 128, page=32, seed=14)
    a, la = run(mt, p, 0.09)
    b, lb = run(mt, p, 0.09)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (16, 1, 128), (3, 3, 96)], ids=lambda h: "x".join(map(str, h)))
def test_chunks_and_single_tokens_in_every_order(mt, heads):
    # tiles with rows in one half and in both follow one another, with growing
    # scores so that reference maxima move
    g = heads[0] // heads[1]
    full = 256 // g  # tokens of a whole tile
    for lens in ([(full, 700), (1, 900), (full + 3, 400), (1, 1), (2, 650), (full, full), (1, 129)],
                 [(1, 513), (2 * full, 2 * full), (1, 256), (full // 2 + 1, 300), (0, 50), (1, 2000)]):
        p = Paged(lens, *heads, page=16, seed=19, q_scale=4.0)
        for kb in p.keys:
            kb *= torch.linspace(0.2, 2.0, len(kb))[:, None, None].to(torch.bfloat16)
        for b, (_, kv) in enumerate(lens):
            for i in range(-(-kv // 16)):
                n = min(16, kv - i * 16)
                p.k[p.pages[b, i], :n] = p.keys[b][i * 16:i * 16 + n]
        compare(mt, p)
        compare(mt, p, window=200, sinks=3)


def test_many_sequences(mt):
    lens = [(1 if b % 7 else 0, (b * 37) % 200 + 1) for b in range(1024)]
    compare(mt, Paged(lens, 4, 2, 64, page=16, seed=15))


def test_many_sequences_with_chunks(mt):
    lens = [(200 + b, 210 + 3 * b) if b % 9 == 0 else (b % 4, 5 * b + 3) for b in range(45)]
    compare(mt, Paged(lens, 8, 2, 64, page=16, seed=21))
    compare(mt, Paged(lens, 8, 2, 64, page=12, seed=21), window=70, sinks=5)


@pytest.mark.parametrize("page", [16, 12], ids=["chunk-kernel", "rows-kernel"])
def test_offsets_beyond_32_bits(mt, page):
    # two pages 2^31 elements apart, V after K in the same allocation
    far = 1 << 31
    p = Paged([(9, 2 * page)], 4, 2, 64, page=page, seed=22, spare=0)
    store = torch.empty(far + 2 * page * 2 * 64, dtype=torch.bfloat16, device="cuda")
    size, strides = (2, page, 2, 64), (far, 128, 64, 1)
    k, v = store.as_strided(size, strides), store.as_strided(size, strides, page * 128)
    k.copy_(p.k)
    v.copy_(p.v)
    q, _, _, pages, q_start, kv_len = p.cuda()
    out, lse = torch.empty_like(q), torch.empty(p.T, 4, device="cuda")
    ws = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, 1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, 9, 0.125, out, ws, lse=lse)
    ref = attention_ref(p, 0.125)
    tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
    check(out, ref[0], tol_out)
    check(lse, ref[1], tol_lse)
    # and the write: the same tokens again, unturned (position 0)
    new = torch.randn(9, 2, 64, device="cuda").to(torch.bfloat16)
    mt.mt_rope_append(q, new, new, torch.zeros(9, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda"), out, k, v, pages,
                      q_start, kv_len)
    for i in range(9):
        at = 2 * page - 9 + i
        pg, r = int(p.pages[0, at // page]), at % page
        assert torch.equal(k[pg, r], new[i]) and torch.equal(v[pg, r], new[i])


def test_long_text_split_over_the_gpu(mt):
    compare(mt, Paged([(1, 20011)], 4, 1, 64, page=16, seed=16))
    compare(mt, Paged([(40, 9000)], 4, 1, 128, page=64, seed=17))


def test_other_stream_and_graph(mt):
    p = Paged([(1, 400), (1, 30)], 8, 2, 128, page=16, seed=18)
    want, wl = run(mt, p, 0.09)
    s = torch.cuda.Stream()
    got, gl = run(mt, p, 0.09, stream=s)
    assert torch.equal(want, got) and torch.equal(wl, gl)
    q, k, v, pages, q_start, kv_len = p.cuda()
    out, lse = torch.zeros_like(q), torch.zeros(p.T, p.hq, device="cuda")
    ws = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, 1, 0.09, out, ws, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, out) and torch.equal(wl, lse)
    # lengths are read on the device: a replay follows them
    p2 = Paged([(1, 200), (1, 30)], 8, 2, 128, page=16, seed=18, width=p.pages.shape[1])
    kv_len.copy_(torch.tensor([200, 30], dtype=torch.int32))
    p.lens, p.kv_len = [(1, 200), (1, 30)], p2.kv_len
    p.keys[0], p.values[0] = p.keys[0][:200], p.values[0][:200]
    graph.replay()
    torch.cuda.synchronize()
    ref = attention_ref(p, 0.09)
    tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
    check(out, ref[0], tol_out)
    check(lse, ref[1], tol_lse)
