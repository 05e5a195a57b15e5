"""GPU tests of mt_cache_keep: every byte of the caches is compared."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    m.mt_device_error(True)
    yield m
    assert m.mt_device_error(True) == 0


class Case:
    def __init__(self, lens, paths, L=2, hkv=2, d=64, page=16, order="nhd", counts=None, cols=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.paths, self.page = lens, paths, page
        need = [-(-max(kv, 0) // page) for _, kv in lens]
        pages = sum(need) + 2
        ids = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[at:at + m]
            at += m
        # any bits, NaN among them
        bits = torch.randint(-2 ** 15, 2 ** 15, (L, 2, pages, page, hkv, d), generator=g).to(torch.int16)
        if order == "hnd":
            self.cache = bits.transpose(3, 4).contiguous().view(torch.bfloat16).cuda().transpose(3, 4)
        elif order == "layers":  # [pages][layer][K, V]
            self.cache = bits.permute(2, 0, 1, 3, 4, 5).contiguous().view(torch.bfloat16).cuda().permute(1, 2, 0, 3, 4, 5)
        else:
            self.cache = bits.view(torch.bfloat16).cuda()
        self.starts = [0]
        for n, _ in lens:
            self.starts.append(self.starts[-1] + n)
        cols = cols or max(1, max(map(len, paths)))
        self.path = torch.full((len(lens), cols), -1, dtype=torch.int32)
        for b, p in enumerate(paths):
            self.path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        self.count = torch.tensor(counts or [len(p) for p in paths], dtype=torch.int32)

    def want(self):
        c = self.cache.contiguous().cpu().view(torch.int16)
        got, news = c.clone(), []
        for b, (n, kv) in enumerate(self.lens):
            base, before, kept = kv - n, -1, 0
            for i in range(min(max(int(self.count[b]), 0), self.path.shape[1])):
                at = int(self.path[b, i])
                if at <= before or at >= n:
                    break
                before, kept = at, kept + 1
                a, z = base + at, base + i
                if z < 0 or at == i:
                    continue
                pa, pz = int(self.table[b, a // self.page]), int(self.table[b, z // self.page])
                if 0 <= pa < c.shape[2] and 0 <= pz < c.shape[2]:
                    got[:, :, pz, z % self.page] = c[:, :, pa, a % self.page]
            news.append(base + kept)
        return got, news

    def check(self, mt, stream=None, whole=False):
        want, news = self.want()
        i32 = dict(dtype=torch.int32, device="cuda")
        new = torch.full((len(self.lens),), 99, **i32)
        args = (self.cache if whole else [(x[0], x[1]) for x in self.cache], self.table.cuda(), torch.tensor(self.starts, **i32),
                torch.tensor([kv for _, kv in self.lens], **i32), self.path.cuda(), self.count.cuda())
        torch.cuda.synchronize()
        mt.mt_cache_keep(*args, new_len=new, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(self.cache.contiguous().cpu().view(torch.int16), want)
        assert new.tolist() == news


@pytest.mark.parametrize("order", ["nhd", "hnd", "layers"])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
def test_paths(mt, page, order):
    lens = [(25, 100), (9, 9), (1, 50), (64, 64), (5, 20), (0, 30), (30, 31)]
    paths = [[0, 3, 4, 9, 24], [0, 1, 2, 8], [0], [0, 2, 4, 6, 8, 10, 12, 60, 61, 62, 63], [], [], [3, 4, 5, 6, 7, 29]]
    Case(lens, paths, page=page, order=order).check(mt)


@pytest.mark.parametrize("order", ["nhd", "hnd", "layers"])
def test_caches_in_one_tensor(mt, order):
    lens, paths = [(25, 100), (9, 9), (64, 64)], [[0, 3, 4, 9, 24], [0, 1, 2, 8], [0, 2, 4, 60, 63]]
    for L in (1, 5, 66):
        Case(lens, paths, L=L, order=order, hkv=3, d=24, seed=L).check(mt, whole=True)


def test_caches_in_one_tensor_that_share_elements(mt):
    c = Case([(12, 40)], [[0, 5, 6]], L=1)
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (c.table.cuda(), torch.tensor(c.starts, **i32), torch.tensor([40], **i32), c.path.cuda(), c.count.cuda())
    shape = c.cache.shape[2:]
    for bad in (c.cache.expand(3, 2, *shape), c.cache[:, :1].expand(1, 2, *shape), c.cache[:, :1].expand(2, 2, *shape)):
        with pytest.raises(mt.MTError) as e:
            mt.mt_cache_keep(bad, *args)
        assert e.value.status == mt.MT_ERR_ALIAS


@pytest.mark.parametrize("hkv,d", [(1, 16), (8, 128), (2, 256), (3, 72), (5, 40), (16, 128)])
def test_heads(mt, hkv, d):
    Case([(25, 100), (12, 40)], [[0, 2, 3, 20], [0, 5, 6, 7, 8, 9, 11]], hkv=hkv, d=d, L=3).check(mt)


@pytest.mark.parametrize("L", [1, 63, 64, 65, 130])
def test_layers(mt, L):
    Case([(12, 40), (7, 19)], [[0, 5, 6], [0, 2, 4, 6]], L=L, d=16).check(mt)


@pytest.mark.parametrize("n", [100, 777])
def test_long_paths(mt, n):
    g = torch.Generator().manual_seed(n)
    every = sorted(torch.randperm(n, generator=g)[:n // 2].tolist())
    Case([(n, n + 13), (n, n)], [every, list(range(n))]).check(mt)
    Case([(n, n + 5)], [list(range(1, n))]).check(mt)  # each token one place on


def test_counts_and_paths_that_end_early(mt):
    lens = [(10, 40)] * 8
    paths = [[0, 2, 2, 3], [0, 5, 4, 6], [0, 2, 10, 11], [-1, 2, 3, 4], [0, 3, 4, 5], [0, 3, 4, 5], [0, 3, 4, 5], [2, 2 ** 31 - 1, 3, 4]]
    Case(lens, paths, counts=[4, 4, 4, 4, 2, -3, 2 ** 31 - 1, 4]).check(mt)


def test_tokens_that_are_not_in_the_cache(mt):
    # more new tokens than the cache has room for: the first positions are negative
    Case([(10, 4), (6, 0), (9, 8)], [[0, 5, 7, 8, 9], [1, 3, 5], [0, 1, 3, 4, 8]]).check(mt)


def test_no_new_lengths(mt):
    c = Case([(12, 40)], [[0, 5, 6]])
    want, _ = c.want()
    i32 = dict(dtype=torch.int32, device="cuda")
    mt.mt_cache_keep([(x[0], x[1]) for x in c.cache], c.table.cuda(), torch.tensor(c.starts, **i32), torch.tensor([40], **i32), c.path.cuda(), c.count.cuda())
    assert torch.equal(c.cache.cpu().view(torch.int16), want)


def test_page_out_of_range_is_reported(mt):
    c = Case([(30, 60), (30, 60)], [[0, 2, 9, 20, 29], [0, 3, 4, 20, 21]])
    c.table[0, 3] = 10000  # holds 48 .. 63
    c.table[1, 2] = -1     # 32 .. 47
    c.check(mt)
    assert mt.mt_device_error(True) == mt.MT_ERR_PAGE


def test_entries_that_are_not_needed_are_not_followed(mt):
    c = Case([(30, 60), (5, 50)], [[0, 2, 3], [0, 1, 2]])
    c.table[0, 0], c.table[0, 3], c.table[1, :] = -1, 99999, -1  # nothing of the second text moves
    c.check(mt)
    assert mt.mt_device_error(False) == 0


def test_many_sequences(mt):
    lens = [(1 + b % 13, 20 + b % 37) for b in range(1024)]
    g = torch.Generator().manual_seed(4)
    paths = [[0] + sorted((1 + torch.randperm(n - 1, generator=g)[:min(n - 1, 4)]).tolist()) if n > 1 else [0] for n, _ in lens]
    Case(lens, paths, d=16).check(mt)


def test_offsets_beyond_32_bits(mt):
    far = 1 << 31
    store = torch.empty(far + 16 * 2 * 2 * 64, dtype=torch.bfloat16, device="cuda")
    k = store.as_strided((2, 16, 2, 64), (far, 128, 64, 1))
    v = store.as_strided((2, 16, 2, 64), (far, 128, 64, 1), 16 * 128)
    i32 = dict(dtype=torch.int32, device="cuda")
    for x in (k, v):
        x.copy_(torch.randn(2, 16, 2, 64, device="cuda"))
    wk, wv = k.clone(), v.clone()
    for i, at in ((1, 9), (2, 19)):
        for x, w in ((k, wk), (v, wv)):
            w[(10 + i) // 16, (10 + i) % 16] = x[(10 + at) // 16, (10 + at) % 16]
    mt.mt_cache_keep([(k, v)], torch.tensor([[0, 1]], **i32), torch.tensor([0, 20], **i32), torch.tensor([30], **i32),
                     torch.tensor([[0, 9, 19]], **i32), torch.tensor([3], **i32))
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_other_stream_and_graph(mt):
    Case([(25, 100)], [[0, 3, 4, 9, 24]]).check(mt, stream=torch.cuda.Stream())
    c = Case([(25, 100), (9, 30)], [[0, 3, 4, 9, 24], [0, 2, 5, 6, 8]])
    i32 = dict(dtype=torch.int32, device="cuda")
    args = [[(x[0], x[1]) for x in c.cache], c.table.cuda(), torch.tensor(c.starts, **i32), torch.tensor([100, 30], **i32), c.path.cuda(),
            torch.zeros(2, **i32)]
    new = torch.zeros(2, **i32)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mt.mt_cache_keep(*args, new_len=new)
    args[5].copy_(c.count)
    want, news = c.want()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.cache.cpu().view(torch.int16), want) and new.tolist() == news
