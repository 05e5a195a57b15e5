"""GPU tests of mt_token_probs against 64-bit probabilities."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    return m


def reference(x, t):
    """[R, V] in 64 bits; t a list of floats."""
    x = x.cpu().double()
    got = torch.zeros_like(x)
    for r in range(x.shape[0]):
        top = x[r].max()  # NaN if any is
        if not bool(top < math.inf):
            got[r] = math.nan
        elif top == -math.inf:
            pass
        elif t[r] > 0:
            e = torch.where(x[r] == -math.inf, 0.0, torch.exp((x[r] - top) / t[r]))
            got[r] = e / e.sum()
        else:
            got[r, int((x[r] == top).nonzero()[0])] = 1.0
    return got


def tolerance(want):
    """Relative to p: an exponential is off by 2^-22 (two steps of exp2f), and 2^-23 in the two
    roundings that take in the rest of its argument; at most two follow one another, in p and in the
    sum: 4 (2^-22 + 2^-23).  The sum's own roundings, V / 512 of them in a thread at the most and 128
    over the threads, and the quotient's."""
    V = want.shape[1]
    return want * (4 * (2.0 ** -22 + 2.0 ** -23) + (V / 512 + 130) * 2.0 ** -24) + 2.0 ** -148


def check(mt, x, t=None, pad=0, out_pad=0, in_place=False, stream=None):
    R, V = x.shape
    rows = torch.full((R, V + pad), 3.0, dtype=x.dtype)
    rows[:, :V] = x
    rows = rows.cuda()
    store = rows if in_place else torch.full((R, V + out_pad), 7.0, device="cuda")
    temps = None if t is None else torch.tensor(t, dtype=torch.float32).cuda()
    torch.cuda.synchronize()
    mt.mt_token_probs(rows[:, :V], store[:, :V], temps, stream=stream)
    torch.cuda.synchronize()
    got = store.cpu()
    assert bool((got[:, V:] == (3.0 if in_place else 7.0)).all()), "columns past the row were written"
    want = reference(x, [1.0] * R if t is None else temps.tolist())
    got = got[:, :V].double()
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(got))
    excess = ((got - want).abs() - tolerance(want))[~nan]
    assert excess.numel() == 0 or float(excess.max()) <= 0, float(excess.max())
    assert bool((got[(x == -math.inf) & ~nan] == 0).all())


DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])


def logits(R, V, dtype, seed=0, scale=3.0):
    return (torch.randn(R, V, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


@DTYPES
@pytest.mark.parametrize("V", [1, 2, 3, 7, 31, 32, 33, 1000, 1024, 1025, 4099, 32000, 50257, 128256, 151936, 262144, 300007])
def test_sizes(mt, dtype, V):
    check(mt, logits(3, V, dtype, V), [1.0, 0.7, 0.0])


@DTYPES
@pytest.mark.parametrize("R,V", [(1, 151936), (9, 5003), (40, 40000), (153, 3001), (700, 517), (2000, 129)])
def test_rows(mt, dtype, R, V):
    check(mt, logits(R, V, dtype, R), [0.3 + 0.01 * (r % 150) for r in range(R)])
    check(mt, logits(R, V, dtype, R))


@DTYPES
@pytest.mark.parametrize("pad,out_pad", [(1, 0), (0, 1), (3, 3), (8, 4), (5, 2)])
def test_strides(mt, dtype, pad, out_pad):
    check(mt, logits(7, 4001, dtype, 5), [1.0] * 7, pad, out_pad)
    check(mt, logits(7, 33000, dtype, 5), [0.5] * 7, pad, out_pad)


@DTYPES
def test_temperatures(mt, dtype):
    t = [0.0, -1.0, math.nan, math.inf, 1e-40, 1e-30, 1e-6, 0.01, 0.1, 1.0, 7.0, 1e6, 1e30, 3e38, -math.inf, -0.0]
    check(mt, logits(len(t), 3000, dtype, 1), t)
    check(mt, logits(len(t), 40000, dtype, 2, scale=20.0), t)


@DTYPES
@pytest.mark.parametrize("V", [50, 1500, 70000])
def test_masks_nan_and_infinities(mt, dtype, V):
    x = logits(12, V, dtype, 3)
    x[0] = -math.inf                       # nothing is left
    x[1] = -math.inf
    x[1, V - 1] = -5.0                     # one token is
    x[2, V // 2] = math.nan
    x[3, 0] = math.inf
    x[4, ::3] = -math.inf
    x[5] = 1.5                             # all alike
    x[6] = -math.inf
    x[7] = torch.finfo(dtype).min
    x[8] = torch.finfo(dtype).min
    x[8, 3] = torch.finfo(dtype).max
    x[9, 1] = math.nan
    x[10, V - 1] = math.nan
    x[10, :V - 1] = -math.inf
    x[11, 5] = math.inf
    x[11, 7] = -math.inf
    check(mt, x, [1.0, 0.5, 1.0, 1.0, 0.8, 1.0, 0.0, 1.0, 1.0, 0.0, 1.0, 0.0])
    check(mt, x[[0, 5, 4, 7, 1, 8]], [0.0] * 6)
    check(mt, x[[0, 5, 4, 7, 1, 8]], [math.inf] * 6)


@DTYPES
def test_the_first_of_equal_logits(mt, dtype):
    for V in (100, 5000, 130000):
        x = logits(6, V, dtype, 7).clamp(max=2.0)
        check(mt, x, [0.0] * 6)
        x[:, V - 2:] = 9.0
        check(mt, x, [0.0] * 6)


def test_in_place(mt):
    for V in (37, 4000, 151936, 300007):
        check(mt, logits(5, V, torch.float32, 4), [1.0, 0.4, 0.0, 2.0, 1.0], pad=3, in_place=True)


@DTYPES
def test_rows_further_apart_than_32_bits(mt, dtype):
    far, V = (1 << 31) + 8, 5000
    x = logits(2, V, dtype, 8)
    rows = torch.empty(far + V, dtype=dtype, device="cuda").as_strided((2, V), (far, 1))
    out = torch.empty(far + V, device="cuda").as_strided((2, V), (far, 1))
    rows.copy_(x)
    mt.mt_token_probs(rows, out)
    want = reference(x, [1.0, 1.0])
    assert bool(((out.cpu().double() - want).abs() <= tolerance(want)).all())


@DTYPES
def test_other_stream_graph_and_equal_runs(mt, dtype):
    x = logits(20, 60000, dtype, 9)
    check(mt, x, [1.0] * 20, stream=torch.cuda.Stream())
    rows, t = x.cuda(), torch.ones(20, device="cuda")
    a, b = torch.empty(20, 60000, device="cuda"), torch.empty(20, 60000, device="cuda")
    mt.mt_token_probs(rows, a, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mt.mt_token_probs(rows, b, t)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    t.fill_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    want = reference(x, [0.5] * 20)
    assert bool(((b.cpu().double() - want).abs() <= tolerance(want)).all())
