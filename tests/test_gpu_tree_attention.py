"""GPU tests of mt_tree_attention against a 64-bit reference: trees of all
sizes, any bits, windows by the row's own position, NaN where no token looks,
pages, layouts, strides, other streams and graphs."""
import math

import pytest
import torch

from paged_util import Paged, attention_bounds, check
from tree_util import bit_rows, mixed_tree, seen_of, tree_attention_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    m.mt_device_error(True)
    yield m
    assert m.mt_device_error(True) == 0


def run(mt, p, seen, scale, window=0, sinks=0, dtype=torch.bfloat16, words=None, max_q=None, out_pad=0, bit_pad=0, stream=None):
    q, k, v, pages, q_start, kv_len = p.cuda()
    words = words or max(1, (p.max_q + 31) // 32)
    store = torch.full((p.T, words + bit_pad), -1, dtype=torch.int32)
    store[:, :words] = bit_rows(seen, p.T, words, fill=-1)
    visible = store.cuda()[:, :words]
    out = torch.full((p.T, p.hq * p.d + out_pad), 7.0, dtype=dtype, device="cuda")
    view = out[:, :p.hq * p.d].unflatten(1, (p.hq, p.d))
    lse = torch.full((p.T, p.hq), 7.0, dtype=torch.float32, device="cuda")
    ws = torch.full((mt.mt_paged_attention_workspace_bytes(p.T, len(p.lens), p.hq, p.hkv, p.d) // 4,), math.nan, device="cuda")
    torch.cuda.synchronize()
    mt.mt_tree_attention(q, k, v, pages, q_start, kv_len, visible, p.max_q if max_q is None else max_q, scale, view, ws, lse=lse,
                         window=window, sinks=sinks, stream=stream)
    torch.cuda.synchronize()
    rows = int(p.q_start[-1])
    assert bool((out[rows:] == 7).all()) and bool((out[:, p.hq * p.d:] == 7).all()), "rows of no sequence were written"
    return view[:rows], lse[:rows]


def compare(mt, p, seen=None, window=0, sinks=0, dtype=torch.bfloat16, rounding=2.0 ** -8, **kw):
    scale = 1.0 / math.sqrt(p.d)
    seen = seen or [seen_of(mixed_tree(n, 3 * b + 1)) for b, (n, _) in enumerate(p.lens)]
    out, lse = run(mt, p, seen, scale, window, sinks, dtype, **kw)
    words = kw.get("words")
    ref = tree_attention_ref(p, [m[:, :32 * words] for m in seen] if words else seen, scale, window, sinks)
    tol_out, tol_lse = attention_bounds(p, ref, rounding if dtype == torch.bfloat16 else 2.0 ** -16, dtype)
    check(lse, ref[1], tol_lse, "lse")
    check(out, ref[0], tol_out, "out")


HEADS = [(4, 4, 64), (8, 2, 128), (14, 2, 64), (3, 1, 96), (6, 2, 72), (16, 1, 128), (2, 2, 16), (5, 5, 128), (8, 1, 256), (40, 8, 40),
         (128, 1, 64), (33, 1, 128)]
KERNELS = pytest.mark.parametrize("page", [16, 12], ids=["chunk-kernel", "rows-kernel"])


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("lens", [[(1, 1)], [(7, 7)], [(25, 403)], [(5, 70), (17, 17), (1, 200), (33, 129)], [(64, 200), (140, 333)]],
                         ids=["one", "alone", "25", "ragged", "large"])
def test_trees(mt, heads, lens):
    compare(mt, Paged(lens, *heads, page=16, seed=1))


@pytest.mark.parametrize("page", [1, 3, 8, 20, 24, 48, 64, 128, 256])
def test_page_sizes(mt, page):
    compare(mt, Paged([(30, 130), (70, 401)], 8, 2, 64, page=page, seed=3))


@pytest.mark.parametrize("base", [0, 1, 31, 32, 33, 63, 64, 96, 97, 127, 128, 129, 250])
@KERNELS
def test_every_offset_of_the_tree_in_a_block(mt, base, page):
    lens = [(n, n + base) for n in (1, 31, 33, 64, 130)]
    compare(mt, Paged(lens, 4, 2, 64, page=page, seed=base))


@KERNELS
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128)], ids=["4x2x64", "8x1x128"])
def test_any_bits(mt, page, heads):
    # rows that see later tokens, themselves or not, nothing at all; every row the same; bits past the sequence's tokens
    g = torch.Generator().manual_seed(5)
    lens = [(40, 100), (3, 3), (150, 290), (9, 9)]
    seen = [torch.rand(n, 160, generator=g) < 0.3 for n, _ in lens]
    seen[0][::5] = False
    seen[1][1] = False
    seen[3][:] = False
    compare(mt, Paged(lens, *heads, page=page, seed=5), seen)
    compare(mt, Paged(lens, *heads, page=page, seed=5), [torch.ones(n, 160, dtype=torch.bool) for n, _ in lens])


@KERNELS
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (20, 300), (64, 4), (100, 70), (1000, 3), (129, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_and_sinks(mt, page, window, sinks):
    for heads in ((8, 2, 128), (7, 1, 64)):
        compare(mt, Paged([(25, 500), (1, 3), (40, 128), (130, 260), (6, 400)], *heads, page=page, seed=5), window=window, sinks=sinks)
    # positions differ within a tile and from tile to tile: a chain, and rows without bits
    lens = [(150, 420), (20, 300)]
    seen = [seen_of(list(range(-1, n - 1))) for n, _ in lens]
    seen[1][::3] = False
    compare(mt, Paged(lens, 4, 2, 64, page=page, seed=6), seen, window=window, sinks=sinks)


@KERNELS
def test_more_new_tokens_than_the_cache_has(mt, page):
    compare(mt, Paged([(40, 25), (6, 0), (3, 1), (0, 30), (70, 64)], 8, 2, 64, page=page, seed=7))


@KERNELS
def test_fewer_words_than_tokens(mt, page):
    # new tokens past the words are seen by none, and their rows see the others
    compare(mt, Paged([(100, 230), (33, 40), (3, 300)], 8, 2, 64, page=page, seed=8), words=1)
    compare(mt, Paged([(1100, 1200)], 2, 1, 64, page=page, seed=8), words=32)


@pytest.mark.parametrize("page", [16, 64, 12])
def test_the_largest_tree(mt, page):
    compare(mt, Paged([(1024, 1100), (1, 50)], 4, 1, 64, page=page, seed=9))


@pytest.mark.parametrize("order", ["hnd", "kv"])
@KERNELS
def test_cache_orders_and_row_strides(mt, order, page):
    compare(mt, Paged([(30, 130), (5, 401)], 8, 2, 128, page=page, order=order, seed=4, q_pad=24, rows_pad=3), out_pad=40, bit_pad=3)


def test_fp32_output(mt):
    for heads in ((8, 2, 128), (14, 2, 64), (8, 1, 256)):
        compare(mt, Paged([(25, 300), (70, 150)], *heads, page=16, seed=9), dtype=torch.float32)


def test_weights_of_the_rows_kernel_are_rounded_to_two_bf16(mt):
    compare(mt, Paged([(9, 900), (20, 300)], 8, 2, 128, page=12, seed=10), rounding=2.0 ** -16)


def test_large_scores(mt):
    compare(mt, Paged([(20, 700), (140, 300)], 8, 2, 64, page=16, seed=11, q_scale=30.0))


@pytest.mark.parametrize("page", [16, 64, 12])
def test_new_tokens_that_none_sees_may_be_nan(mt, page):
    # padding in the tree: no row's bit, infinities and NaN in the cache
    lens = [(40, 100), (64, 190), (150, 300)]
    p = Paged(lens, 8, 2, 64, page=page, seed=23)
    g = torch.Generator().manual_seed(3)
    seen = []
    for b, (n, kv) in enumerate(lens):
        m = seen_of(mixed_tree(n, b))
        out = torch.rand(n, generator=g) < 0.4
        out[0] = False
        m[:, out] = False
        seen.append(m)
        for j in out.nonzero()[:, 0].tolist():
            at = kv - n + j
            for x, bad in ((p.k, math.nan), (p.v, math.nan if j % 2 else math.inf)):
                x[p.pages[b, at // page], at % page] = bad
    compare(mt, p, seen)
    compare(mt, p, seen, window=50, sinks=3)


@pytest.mark.parametrize("page", [16, 64, 12])
def test_keys_before_every_rows_window_may_be_nan(mt, page):
    # every row sees at least `low` new tokens: nothing up to base + low - 1 - window is seen
    low, window, sinks = 6, 40, 2
    lens = [(20, 200), (70, 330)]
    p = Paged(lens, 8, 2, 64, page=page, seed=25)
    seen = []
    for b, (n, kv) in enumerate(lens):
        m = seen_of(mixed_tree(n, b))
        m[:, :low] = True
        seen.append(m)
        for j in range(sinks, kv - n + low - window):
            for x, bad in ((p.k, math.nan), (p.v, math.inf if j % 2 else math.nan)):
                x[p.pages[b, j // page], j % page] = bad
    compare(mt, p, seen, window=window, sinks=sinks)


def test_pages_that_no_token_sees_are_not_followed(mt):
    p = Paged([(30, 900)], 8, 2, 64, page=16, seed=12)
    first = (870 - 100 + 1) // 16
    p.pages[0, 1:first] = -1
    compare(mt, p, window=100, sinks=5)
    assert mt.mt_device_error(False) == 0


@KERNELS
def test_page_out_of_range_is_reported(mt, page):
    p = Paged([(30, 100)], 4, 2, 64, page=page, seed=13)
    p.pages[0, 2] = p.num_pages
    p.keys[0][2 * page:3 * page] = 0
    p.values[0][2 * page:3 * page] = 0
    seen = [seen_of(mixed_tree(30, 1))]
    out, lse = run(mt, p, seen, 0.125)
    assert mt.mt_device_error(True) == mt.MT_ERR_PAGE
    ref = tree_attention_ref(p, seen, 0.125)
    tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
    check(out, ref[0], tol_out)
    check(lse, ref[1], tol_lse)


def test_a_chain_is_a_chunk(mt):
    # the same tokens by mt_paged_attention, within the bounds of the same reference
    for heads, page in (((8, 2, 128), 16), ((14, 2, 64), 16), ((8, 2, 64), 12)):
        lens = [(40, 300), (1, 700), (130, 130), (3, 9)]
        p = Paged(lens, *heads, page=page, seed=14)
        out, lse = run(mt, p, [seen_of(list(range(-1, n - 1))) for n, _ in lens], 0.09)
        ref = tree_attention_ref(p, [torch.tril(torch.ones(n, n, dtype=torch.bool)) for n, _ in lens], 0.09)
        tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
        check(out, ref[0], tol_out)
        check(lse, ref[1], tol_lse)
        q, k, v, pages, q_start, kv_len = p.cuda()
        other, ol = torch.empty_like(q), torch.empty(p.T, heads[0], device="cuda")
        ws = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, len(lens), *heads), dtype=torch.uint8, device="cuda")
        mt.mt_paged_attention(q, k, v, pages, q_start, kv_len, p.max_q, 0.09, other, ws, lse=ol)
        check(other, ref[0], tol_out)
        check(ol, ref[1], tol_lse)


@pytest.mark.parametrize("lens", [[(16, 5000)] * 3, [(70, 3000), (1, 4000), (33, 1500)], [(300, 2500)]], ids=["small", "mixed", "large"])
def test_two_calls_give_the_same_bits(mt, lens):
    p = Paged(lens, 8, 2, 128, page=32, seed=14)
    seen = [seen_of(mixed_tree(n, b)) for b, (n, _) in enumerate(lens)]
    a, la = run(mt, p, seen, 0.09)
    b, lb = run(mt, p, seen, 0.09)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (16, 1, 128), (3, 3, 96)], ids=lambda h: "x".join(map(str, h)))
def test_trees_of_every_size_one_after_another(mt, heads):
    g = heads[0] // heads[1]
    full = 256 // g
    for lens in ([(full, 700), (1, 900), (full + 3, 400), (1, 1), (2, 650), (full, full), (1, 129)],
                 [(1, 513), (2 * full, 2 * full), (1, 256), (full // 2 + 1, 300), (0, 50), (1, 2000)]):
        compare(mt, Paged(lens, *heads, page=16, seed=19, q_scale=2.0))
        compare(mt, Paged(lens, *heads, page=16, seed=19, q_scale=2.0), window=200, sinks=3)


def test_many_sequences(mt):
    lens = [(b % 9, (b * 37) % 200 + 9) for b in range(1024)]
    compare(mt, Paged(lens, 4, 2, 64, page=16, seed=15))


def test_long_texts_split_over_the_gpu(mt):
    compare(mt, Paged([(16, 20011)], 4, 1, 64, page=16, seed=16))
    compare(mt, Paged([(40, 9000)], 4, 1, 128, page=64, seed=17))


@KERNELS
def test_offsets_beyond_32_bits(mt, page):
    far = 1 << 31
    p = Paged([(9, 2 * page)], 4, 2, 64, page=page, seed=22, spare=0)
    store = torch.empty(far + 2 * page * 2 * 64, dtype=torch.bfloat16, device="cuda")
    size, strides = (2, page, 2, 64), (far, 128, 64, 1)
    k, v = store.as_strided(size, strides), store.as_strided(size, strides, page * 128)
    k.copy_(p.k)
    v.copy_(p.v)
    q, _, _, pages, q_start, kv_len = p.cuda()
    # the rows of bits as far apart
    seen = [seen_of(mixed_tree(9, 1))]
    bits = torch.empty(8 * (far // 8) + 1, dtype=torch.int32, device="cuda").as_strided((9, 1), (far // 8, 1))
    bits.copy_(bit_rows(seen, 9, 1))
    out, lse = torch.empty_like(q), torch.empty(p.T, 4, device="cuda")
    ws = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, 1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    mt.mt_tree_attention(q, k, v, pages, q_start, kv_len, bits, 9, 0.125, out, ws, lse=lse)
    ref = tree_attention_ref(p, seen, 0.125)
    tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
    check(out, ref[0], tol_out)
    check(lse, ref[1], tol_lse)


def test_other_stream_and_graph(mt):
    lens = [(20, 400), (9, 30)]
    p = Paged(lens, 8, 2, 128, page=16, seed=18)
    seen = [seen_of(mixed_tree(n, b)) for b, (n, _) in enumerate(lens)]
    want, wl = run(mt, p, seen, 0.09)
    got, gl = run(mt, p, seen, 0.09, stream=torch.cuda.Stream())
    assert torch.equal(want, got) and torch.equal(wl, gl)
    q, k, v, pages, q_start, kv_len = p.cuda()
    bits = bit_rows(seen, p.T, 1).cuda()
    out, lse = torch.zeros_like(q), torch.zeros(p.T, p.hq, device="cuda")
    ws = torch.empty(mt.mt_paged_attention_workspace_bytes(p.T, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mt.mt_tree_attention(q, k, v, pages, q_start, kv_len, bits, 20, 0.09, out, ws, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, out) and torch.equal(wl, lse)
    # bits and lengths are read on the device: a replay follows them
    seen = [seen_of(mixed_tree(20, 9)), seen_of([-1] * 9)]
    bits.copy_(bit_rows(seen, p.T, 1))
    kv_len.copy_(torch.tensor([200, 30], dtype=torch.int32))
    p.lens, p.kv_len = [(20, 200), (9, 30)], kv_len.cpu()
    p.keys[0], p.values[0] = p.keys[0][:200], p.values[0][:200]
    graph.replay()
    torch.cuda.synchronize()
    ref = tree_attention_ref(p, seen, 0.09)
    tol_out, tol_lse = attention_bounds(p, ref, 2.0 ** -8, torch.bfloat16)
    check(out, ref[0], tol_out)
    check(lse, ref[1], tol_lse)


@pytest.mark.parametrize("max_q", [1, 1000])
def test_the_hint_changes_no_result(mt, max_q):
    compare(mt, Paged([(30, 130), (90, 401), (1, 1)], 8, 2, 64, page=16, seed=6), max_q=max_q)
