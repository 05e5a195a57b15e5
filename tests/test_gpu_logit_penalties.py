"""GPU tests of mt_logit_penalties against a 64-bit reference: types, odd
vocabularies and strides, histories with padding and repeats, repeated bias
entries, masks that leave nothing, non-finite logits."""
import math

import pytest
import torch

from paged_util import HALF, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    m.mt_device_error(True)
    yield m
    assert m.mt_device_error(True) == 0


def ragged(rows, dtype):
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + len(r))
    flat = [x for r in rows for x in r]
    return torch.tensor(flat, dtype=dtype), torch.tensor(starts, dtype=torch.int32)


def reference(x, hist, prompt, rep, pres, freq, bias, allowed):
    y, size = x.double().clone(), x.double().abs()
    V = x.shape[1]
    for b in range(x.shape[0]):
        for t, val in dict(bias[b]).items():
            y[b, t] += torch.tensor(val, dtype=torch.float32).double()
            size[b, t] += abs(val)
        known = sorted({t for t in hist[b] if 0 <= t < V})
        for t in known:
            y[b, t] = y[b, t] / rep[b] if y[b, t] > 0 else y[b, t] * rep[b]
            size[b, t] *= max(float(rep[b]), 1 / float(rep[b]))
            n = hist[b][prompt[b]:].count(t)
            if n:
                y[b, t] -= freq[b] * n + pres[b]
                size[b, t] += abs(float(freq[b])) * n + abs(float(pres[b]))
        if allowed is not None:
            y[b, ~allowed[b]] = -math.inf
    return y, size


def words(allowed):
    B, V = allowed.shape
    n = (V + 31) // 32
    bits = torch.zeros(B, n * 32, dtype=torch.int64)
    bits[:, :V] = allowed.long()
    w = (bits.view(B, n, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def case(mt, B, V, dtype, n_hist=30, n_bias=6, mask=True, in_place=False, pad=0, offset=0, seed=0, logits=None, params=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda n, hi: torch.randint(0, hi, (n,), generator=g).tolist()  # noqa: E731
    x = (torch.randn(B, V, generator=g) * 4).to(dtype) if logits is None else logits.to(dtype)
    # ids out of range pad the histories; few distinct ids: repeats
    hist = [[(t if i % 9 else -1) if i % 11 else V + 3 for i, t in enumerate(r(n_hist * (b + 1) // B, max(1, V // 3)))] for b in range(B)]
    prompt = [min(len(h), len(h) // 2 + b % 2) for b, h in enumerate(hist)]
    bias = [list(zip(r(n_bias, V) + r(2, min(V, 3)), (torch.randn(n_bias + 2, generator=g) * 3).tolist())) for _ in range(B)]
    rep = 1 + 0.4 * torch.rand(B, generator=g)
    pres, freq = torch.rand(B, generator=g), torch.rand(B, generator=g) - 0.3
    allowed = torch.rand(B, V, generator=g) < 0.5 if mask else None
    if mask and B > 1:
        allowed[1] = False  # a grammar that leaves nothing
    if not params:
        rep, pres, freq = torch.ones(B), torch.zeros(B), torch.zeros(B)
    rows = torch.full((B, V + pad + offset), 9.0, dtype=dtype, device="cuda")
    src = rows[:, offset:offset + V]
    src.copy_(x)
    dst = src if in_place else torch.full((B, V + pad + offset), 7.0, dtype=dtype, device="cuda")[:, offset:offset + V]
    h, hs = ragged(hist, torch.int32)
    ids, bs = ragged([[t for t, _ in row] for row in bias], torch.int32)
    vals = torch.tensor([w for row in bias for _, w in row], dtype=torch.float32)
    up = lambda t: t.cuda()  # noqa: E731
    kw = dict(repetition=up(rep), presence=up(pres), frequency=up(freq)) if params else {}
    torch.cuda.synchronize()
    mt.mt_logit_penalties(src, dst, history=up(h), history_start=up(hs), prompt_len=up(torch.tensor(prompt, dtype=torch.int32)),
                          bias_ids=up(ids), bias_values=up(vals), bias_start=up(bs), allowed=up(words(allowed)) if mask else None, **kw)
    torch.cuda.synchronize()
    want, size = reference(x, hist, prompt, rep.double(), pres.double(), freq.double(), bias, allowed)
    # what the type cannot hold rounds to infinity
    top = torch.finfo(dtype).max * (1 + HALF[dtype])
    want = torch.where(want.abs() > top, want.sign() * math.inf, want)
    # bias sum, quotient, product and two differences in fp32, then the output's rounding
    tol = HALF[dtype] * want.abs().nan_to_num(posinf=0) + 8 * 2.0 ** -24 * size.nan_to_num(posinf=0, nan=0) + 1e-30
    got = dst.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    check(got.nan_to_num(nan=0.0, posinf=math.inf, neginf=-math.inf), want.nan_to_num(nan=0.0, posinf=math.inf, neginf=-math.inf), tol)
    if not in_place and pad + offset:
        base = dst._base if dst._base is not None else dst
        assert bool((base[:, :offset] == 7).all()) and bool((base[:, offset + V:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 7, 32, 33, 1000, 2047, 2048, 2049, 8199, 50257])
def test_vocabularies(mt, V, dtype):
    case(mt, 3, V, dtype, n_hist=200, n_bias=min(V, 20))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 0), (0, 1), (5, 2), (8, 8)])
def test_strides_and_alignment(mt, pad, offset, dtype):
    case(mt, 4, 4001, dtype, pad=pad, offset=offset, seed=1)
    case(mt, 4, 4001, dtype, pad=pad, offset=offset, in_place=True, seed=2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_many_rows(mt, dtype):
    # beyond the few-sequences case: larger blocks
    case(mt, 48, 150001, dtype, n_hist=300, seed=3)


def test_no_options(mt):
    x = torch.randn(2, 777, device="cuda")
    out = torch.empty_like(x)
    mt.mt_logit_penalties(x, out)
    assert torch.equal(x, out)
    case(mt, 2, 777, torch.float32, mask=False, params=False)
    case(mt, 2, 777, torch.bfloat16, n_hist=0, n_bias=0, seed=4)


def test_long_history(mt):
    case(mt, 2, 5000, torch.float32, n_hist=70000, seed=5)


def test_bias_of_one_token_given_often(mt):
    # the last entry counts, whatever order the entries are met in
    V = 100
    x = torch.zeros(1, V, device="cuda")
    ids = torch.full((5000,), 42, dtype=torch.int32, device="cuda")
    vals = torch.arange(5000, dtype=torch.float32, device="cuda")
    out = torch.empty_like(x)
    mt.mt_logit_penalties(x, out, bias_ids=ids, bias_values=vals, bias_start=torch.tensor([0, 5000], dtype=torch.int32, device="cuda"))
    want = torch.zeros(1, V)
    want[0, 42] = 4999
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_non_finite_logits(mt, dtype):
    x = torch.randn(2, 999, generator=torch.Generator().manual_seed(6))
    x[:, ::7] = math.inf
    x[:, 1::7] = -math.inf
    x[0, 2::7] = math.nan
    x[:, 3::7] = torch.finfo(dtype).min
    case(mt, 2, 999, dtype, n_hist=400, logits=x, seed=7)


def test_two_calls_give_the_same_bits_and_a_graph(mt):
    V = 20011
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(3, V, device="cuda", generator=g)
    h = torch.randint(0, 50, (6000,), device="cuda", generator=g, dtype=torch.int32)
    hs = torch.tensor([0, 2000, 2000, 6000], dtype=torch.int32, device="cuda")
    par = torch.tensor([1.2, 1.1, 1.3], device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    call = lambda o: mt.mt_logit_penalties(x, o, history=h, history_start=hs, repetition=par, presence=par, frequency=par)  # noqa: E731
    call(a)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
