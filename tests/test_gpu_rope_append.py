"""GPU tests of mt_rope_append against a 64-bit reference: axes, pairings,
partial rotation, norms, far and negative positions, cache orders, tokens
without a place."""
import math

import pytest
import torch

from paged_util import HALF, Paged, check

pytestmark = pytest.mark.gpu

# fp32 steps between the input and the rounding of an element: the mean square
# (256 products in a butterfly at most), its root, the gain, two products and
# a sum, the sine's and cosine's own error and the angle's 2^-25 of half a turn
FP32 = 64 * 2.0 ** -24


@pytest.fixture(scope="module")
def mt():
    import quantized_gemv_epilogues_gb300 as m
    torch.cuda.set_device(0)
    m.mt_device_error(True)
    yield m
    assert m.mt_device_error(True) == 0


def turned(x, angle, weight, eps, adjacent):
    """(result, size): size bounds what an element's rotation adds up."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
    rot = 2 * angle.shape[1]
    y, size = x.clone(), x.abs()
    ia, ib = (torch.arange(0, rot, 2), torch.arange(1, rot, 2)) if adjacent else (torch.arange(rot // 2), torch.arange(rot // 2, rot))
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    both = x[..., ia].abs() + x[..., ib].abs()
    size = size.clone()
    size[..., ia] = both
    size[..., ib] = both
    return y, size


def case(mt, lens, hq, hkv, d, page=16, order="nhd", rot=None, axes=1, adjacent=False, norm=False, in_place=False, base=0, seed=0,
         use_axis=True, theta=10000.0, one_gain=False):
    p = Paged(lens, hq, hkv, d, page, order=order, seed=seed, rows_pad=2)
    g = torch.Generator().manual_seed(seed + 100)
    T, rot = p.T, rot or d // 16 * 16
    qkv = torch.randn(T, (hq + 2 * hkv) * d + 8, generator=g).to(torch.bfloat16)
    inv_freq = (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
    pos = torch.randint(-50, 3000, (axes, T), generator=g, dtype=torch.int32) + base
    axis = (torch.arange(rot // 2) % axes).to(torch.uint8) if use_axis else None
    qn = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm else None
    kn = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm and not one_gain else None
    eps = 1e-5

    dev = qkv.cuda()
    q, k, v = dev[:, :(hq + 2 * hkv) * d].split([hq * d, hkv * d, hkv * d], 1)
    q, k, v = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
    out = q if in_place else torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _, kc, vc, pages, q_start, kv_len = p.cuda()
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    args = [up(t) for t in (pos if axes > 1 else pos[0], inv_freq, axis, qn, kn)]
    torch.cuda.synchronize()
    mt.mt_rope_append(q, k, v, args[0], args[1], out, kc, vc, pages, q_start, kv_len, axis=args[2], q_norm=args[3], k_norm=args[4],
                      eps=eps, pairing=mt.MT_ROPE_ADJACENT if adjacent else mt.MT_ROPE_HALF)
    torch.cuda.synchronize()

    rows = int(p.q_start[-1])
    which = torch.arange(rot // 2) % axes if use_axis else torch.zeros(rot // 2, dtype=torch.long)
    angle = pos[which].t().double() * inv_freq.double()
    hq_, hk_, hv_ = qkv[:, :(hq + 2 * hkv) * d].split([hq * d, hkv * d, hkv * d], 1)
    rq, sq = turned(hq_.unflatten(1, (hq, d)), angle, qn, eps, adjacent)
    rk, sk = turned(hk_.unflatten(1, (hkv, d)), angle, kn, eps, adjacent)
    tol = lambda r, s: HALF[torch.bfloat16] * r.abs() + 2 * FP32 * s + 1e-30  # noqa: E731
    check(out[:rows], rq[:rows], tol(rq, sq)[:rows], "q")
    if in_place:
        assert torch.equal(out[rows:].cpu(), hq_.unflatten(1, (hq, d))[rows:])
    else:
        assert bool((out[rows:] == 7).all()), "rows of no sequence were written"
    # the caches: the new tokens' slots, and nothing else
    want_k, tol_k = p.k.double().clone(), torch.zeros_like(p.k, dtype=torch.float64)
    want_v = p.v.clone()
    for b, (n, kv) in enumerate(lens):
        for i in range(n):
            at, t = kv - n + i, int(p.q_start[b]) + i
            if at < 0:
                continue
            pg, r = int(p.pages[b, at // page]), at % page
            want_k[pg, r], tol_k[pg, r] = rk[t], tol(rk, sk)[t]
            want_v[pg, r] = hv_.unflatten(1, (hkv, d))[t]
    got_k, got_v = kc.cpu().contiguous(), vc.cpu().contiguous()
    assert torch.equal(torch.isnan(got_k), torch.isnan(want_k)) and torch.equal(torch.isnan(got_v), torch.isnan(want_v))
    check(torch.nan_to_num(got_k.double()), torch.nan_to_num(want_k), tol_k, "k_cache")
    assert torch.equal(torch.nan_to_num(got_v), torch.nan_to_num(want_v))


LENS = [(1, 40), (5, 5), (0, 9), (18, 50), (1, 1)]


@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (3, 1, 96), (6, 2, 72), (2, 2, 16), (4, 1, 256), (40, 8, 80)],
                         ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("adjacent", [False, True], ids=["half", "adjacent"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
def test_heads(mt, heads, adjacent, norm):
    case(mt, LENS, *heads, adjacent=adjacent, norm=norm, axes=3)


@pytest.mark.parametrize("rot", [16, 32, 64, 112, 128])
@pytest.mark.parametrize("adjacent", [False, True], ids=["half", "adjacent"])
def test_partial_rotation(mt, rot, adjacent):
    case(mt, LENS, 4, 2, 128, rot=rot, adjacent=adjacent, norm=True, seed=1)
    case(mt, LENS, 4, 2, 256, rot=rot, adjacent=adjacent, seed=1)


@pytest.mark.parametrize("base", [1 << 20, (1 << 30) - 4000, -(1 << 30)])
def test_far_positions(mt, base):
    case(mt, LENS, 4, 2, 64, axes=2, base=base, seed=2)


@pytest.mark.parametrize("theta", [1.0, 500.0, 5e6, 1e-3])
def test_frequencies_of_every_size(mt, theta):
    # 1: a radian a step for every pair; below 1: frequencies above one
    case(mt, LENS, 4, 2, 64, theta=theta, seed=3)


@pytest.mark.parametrize("order,page", [("hnd", 16), ("kv", 3), ("nhd", 1), ("nhd", 100)])
def test_cache_orders(mt, order, page):
    case(mt, LENS, 4, 2, 64, order=order, page=page, axes=2, seed=4)


def test_in_place_and_one_gain(mt):
    case(mt, LENS, 4, 2, 64, in_place=True, axes=4, norm=True, seed=5)
    case(mt, LENS, 4, 2, 64, norm=True, one_gain=True, use_axis=False, seed=6)


def test_tokens_without_a_place(mt):
    case(mt, [(6, 4), (1, 0), (3, 3)], 4, 2, 64, seed=7)


def test_many_tokens(mt):
    case(mt, [(1300, 1300), (1, 77), (37, 300)], 4, 2, 64, axes=3, norm=True, seed=8)
    case(mt, [(1, b % 50 + 1) for b in range(700)], 4, 2, 128, axes=2, seed=9)


@pytest.mark.parametrize("adjacent,norm,order", [(False, True, "hnd"), (True, False, "kv")])
def test_thousands_of_tokens(mt, adjacent, norm, order):
    lens = [(700, 760), (0, 3), (1, 1), (233, 200), (379, 380)] + [(1, 17 + b) for b in range(40)]
    case(mt, lens, 4, 2, 64, adjacent=adjacent, norm=norm, order=order, page=24, axes=3, seed=11)
    case(mt, [(7900, 7900), (3, 9)], 3, 1, 32, adjacent=adjacent, norm=norm, order=order, page=24, axes=2, seed=12)


def test_page_out_of_range_is_reported(mt):
    p = Paged([(3, 20)], 4, 2, 64, 16, seed=10)
    q, kc, vc, pages, q_start, kv_len = p.cuda()
    pages[0, 1] = -1
    before = kc.clone(), vc.clone()
    kv = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    freq = torch.ones(32, device="cuda")
    mt.mt_rope_append(q, kv, kv, torch.zeros(3, dtype=torch.int32, device="cuda"), freq, out, kc, vc, pages, q_start, kv_len)
    torch.cuda.synchronize()
    assert mt.mt_device_error(True) == mt.MT_ERR_PAGE
    assert torch.equal(torch.nan_to_num(kc), torch.nan_to_num(before[0])) and torch.equal(torch.nan_to_num(vc), torch.nan_to_num(before[1]))
    assert torch.equal(out, q)  # position 0 turns nothing
