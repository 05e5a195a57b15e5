"""Refusals of the calls around the projections (no device needed: arguments
are checked before anything is launched), and the host-side model of the
rotary angle's integer arithmetic."""
import ctypes
import math
import os
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, GROUP, ALIGN, FORMAT, ALIAS = 0, 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def mt():
    import __graft_entry__
    __graft_entry__._libbuild().build()
    import quantized_gemv_epilogues_gb300 as m
    return m


def A(i):
    """The i-th fake device address: 16-byte aligned, far from the others, never dereferenced."""
    return (i + 1) << 36


def cache(mt, **kw):
    d = dict(k=A(0), v=A(1), page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64, num_pages=10, page_size=16, kv_heads=2,
             head_dim=64)
    d.update(kw)
    return mt.PagedCache(*[d[n] for n, _ in mt.PagedCache._fields_])


def batch(mt, **kw):
    d = dict(q_start=A(2), kv_len=A(3), pages=A(4), pages_ld=4, B=3, T=5, max_pages=4, max_q=2)
    d.update(kw)
    return mt.PagedBatch(*[d[n] for n, _ in mt.PagedBatch._fields_])


def attention(mt, c=None, b=None, **kw):
    d = dict(q=A(5), q_stride=256, q_heads=4, scale=0.1, window=0, sinks=0, out=A(6), out_stride=256, dtype=0, lse=A(7), ws=A(8),
             ws_bytes=1 << 30)
    d.update(kw)
    c, b = c or cache(mt), b or batch(mt)
    return mt.raw("mt_paged_attention")(d["q"], d["q_stride"], d["q_heads"], ctypes.byref(c), ctypes.byref(b), d["scale"], d["window"],
                                        d["sinks"], d["out"], d["out_stride"], d["dtype"], d["lse"], d["ws"], d["ws_bytes"], None)


def rope(mt, c=None, b=None, **kw):
    d = dict(q=A(5), q_stride=256, k=A(6), k_stride=128, v=A(7), v_stride=128, q_heads=4, q_norm=None, k_norm=None, eps=1e-6,
             positions=A(8), n_axes=3, inv_freq=A(9), axis=None, rot=64, pairing=0, q_out=A(10), q_out_stride=256)
    d.update(kw)
    c, b = c or cache(mt), b or batch(mt)
    return mt.raw("mt_rope_append")(*[d[n] for n in ("q", "q_stride", "k", "k_stride", "v", "v_stride", "q_heads", "q_norm", "k_norm", "eps",
                                                     "positions", "n_axes", "inv_freq", "axis", "rot", "pairing", "q_out", "q_out_stride")],
                                    ctypes.byref(c), ctypes.byref(b), None)


def logits(mt, **kw):
    d = dict(logits=A(0), ld=1000, out=A(1), out_ld=1000, dtype=1, B=2, V=1000, history=A(2), history_start=A(3), prompt_len=A(4),
             n_history=50, repetition=A(5), presence=A(6), frequency=A(7), bias_ids=A(8), bias_values=A(9), bias_start=A(10), n_bias=5,
             allowed=A(11), allowed_ld=32)
    d.update(kw)
    return mt.raw("mt_logit_penalties")(*d.values(), None)


BAD_CACHE = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(k=A(0) + 8), ALIGN), (dict(num_pages=0), SHAPE), (dict(page_size=0), SHAPE),
             (dict(page_size=65537), SHAPE), (dict(kv_heads=0), SHAPE), (dict(head_dim=8), SHAPE), (dict(head_dim=60), SHAPE),
             (dict(head_dim=264), SHAPE), (dict(token_stride=130), ALIGN), (dict(token_stride=32), SHAPE), (dict(head_stride=-64), SHAPE),
             (dict(page_stride=0), SHAPE)]
BAD_BATCH = [(dict(q_start=None), NULL), (dict(kv_len=None), NULL), (dict(pages=None), NULL), (dict(B=0), SHAPE), (dict(B=1025), SHAPE),
             (dict(T=-1), SHAPE), (dict(T=(1 << 22) + 1), SHAPE), (dict(max_pages=0), SHAPE), (dict(pages_ld=3), SHAPE),
             (dict(max_pages=1 << 27, pages_ld=1 << 27), SHAPE), (dict(kv_len=A(3) + 2), ALIGN)]


@pytest.mark.parametrize("call", [attention, rope], ids=["attention", "rope"])
def test_cache_and_batch_refusals(mt, call):
    for kw, want in BAD_CACHE:
        assert call(mt, c=cache(mt, **kw)) == want, kw
    for kw, want in BAD_BATCH:
        assert call(mt, b=batch(mt, **kw)) == want, kw
    assert call(mt, b=batch(mt, T=0)) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL), (dict(dtype=2), FORMAT), (dict(q_heads=0), SHAPE),
    (dict(q_heads=5), SHAPE), (dict(q_heads=512, q_stride=1 << 20, out_stride=1 << 20), SHAPE), (dict(q_stride=248), SHAPE),
    (dict(out_stride=128), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=math.inf), SHAPE),
    (dict(scale=math.nan), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(q_stride=260), ALIGN),
    (dict(q=A(5) + 8), ALIGN), (dict(out=A(6) + 2), ALIGN), (dict(ws=A(8) + 8), ALIGN), (dict(lse=A(7) + 2), ALIGN),
    (dict(ws_bytes=100), SHAPE), (dict(out=A(5)), ALIAS), (dict(out=A(0)), ALIAS), (dict(lse=A(6)), ALIAS), (dict(ws=A(5)), ALIAS),
    (dict(out=A(4)), ALIAS)], ids=str)
def test_attention_refusals(mt, kw, want):
    assert attention(mt, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(positions=None), NULL), (dict(inv_freq=None), NULL),
    (dict(q_out=None), NULL), (dict(pairing=2), FORMAT), (dict(q_heads=0), SHAPE), (dict(q_heads=1025, q_stride=1 << 20), SHAPE),
    (dict(n_axes=0), SHAPE), (dict(n_axes=9), SHAPE), (dict(rot=0), SHAPE), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE),
    (dict(q_stride=128), SHAPE), (dict(k_stride=64), SHAPE), (dict(v_stride=64), SHAPE), (dict(q_out_stride=64), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=math.nan), SHAPE), (dict(k_stride=132), ALIGN), (dict(k=A(6) + 8), ALIGN),
    (dict(q_norm=A(11) + 2), ALIGN), (dict(positions=A(8) + 1), ALIGN), (dict(q_out=A(5) + 64), ALIAS),
    (dict(q_out=A(5), q_out_stride=512), ALIAS), (dict(q_out=A(6)), ALIAS), (dict(k=A(0)), ALIAS), (dict(q_out=A(1)), ALIAS),
    (dict(q_out=A(9)), ALIAS)], ids=str)
def test_rope_refusals(mt, kw, want):
    assert rope(mt, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), NULL), (dict(out=None), NULL), (dict(dtype=2), FORMAT), (dict(history=None), NULL), (dict(history_start=None), NULL),
    (dict(history=None, history_start=None), NULL), (dict(bias_ids=None), NULL), (dict(bias_start=None), NULL), (dict(bias_values=None), NULL),
    (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(V=0), SHAPE), (dict(V=(1 << 24) + 1, ld=1 << 25, out_ld=1 << 25), SHAPE),
    (dict(ld=999), SHAPE), (dict(out_ld=999), SHAPE), (dict(n_history=-1), SHAPE), (dict(n_bias=-1), SHAPE), (dict(allowed_ld=31), SHAPE),
    (dict(logits=A(0) + 2), ALIGN), (dict(history=A(2) + 2), ALIGN), (dict(allowed=A(11) + 1), ALIGN), (dict(out=A(0) + 400), ALIAS),
    (dict(out=A(0), out_ld=2000), ALIAS), (dict(out=A(11)), ALIAS), (dict(out=A(2)), ALIAS)], ids=str)
def test_logit_refusals(mt, kw, want):
    assert logits(mt, **kw) == want


def test_nothing_to_do(mt):
    assert logits(mt, B=0) == OK
    assert logits(mt, B=0, logits=None, out=None) == OK
    assert attention(mt, b=batch(mt, T=0), q=None, out=None, ws=None, lse=None) == OK


def test_status_string_of_a_bad_page(mt):
    assert mt.mt_status_string(mt.MT_ERR_PAGE).startswith("MT_ERR_PAGE")


def test_python_refusals(mt):
    import torch
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    pages, start, kv = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32), torch.tensor([2], dtype=torch.int32)
    out, ws = torch.zeros_like(q), torch.zeros(64, dtype=torch.uint8)
    good = dict(q=q, k_cache=c, v_cache=c, pages=pages, q_start=start, kv_len=kv, max_q=2, scale=0.1, out=out, workspace=ws, stream=0)
    for kw, err in ((dict(q=q.float()), TypeError), (dict(pages=pages.long()), TypeError), (dict(q_start=kv), ValueError),
                    (dict(v_cache=c[:2]), ValueError), (dict(out=out[:1]), ValueError), (dict(q=q[:, :, :32]), ValueError),
                    (dict(out=out.half()), TypeError), (dict(kv_len=torch.zeros(2, dtype=torch.int32)), ValueError),
                    (dict(k_cache=c.transpose(2, 3), v_cache=c.transpose(2, 3)), ValueError)):
        with pytest.raises(err):
            mt.mt_paged_attention(**{**good, **kw})
    with pytest.raises(mt.MTError):  # the workspace is too small
        mt.mt_paged_attention(**good)


def turn_fraction(m, e):
    """The kernel's F for f = m 2^e: 64 fraction bits of f / 2 pi, truncated, from 128 bits of 1 / 2 pi."""
    c = 0x28BE60DB9391054A7F09D5F47D4D3770
    sh = 64 - e
    return ((m * c) >> sh if sh >= 0 else 0) & (2 ** 64 - 1)


def test_angle_arithmetic_against_rationals():
    # 200 digits of 2 pi by Machin's formula
    def arctan_inv(n, digits):
        one = 10 ** (digits + 10)
        x = s = one // n
        k, sign = 1, -1
        while x:
            x //= n * n
            k += 2
            s += sign * (x // k)
            sign = -sign
        return Fraction(s, one)
    two_pi = 8 * (4 * arctan_inv(5, 200) - arctan_inv(239, 200))
    assert int(Fraction(2 ** 128) / two_pi) == 0x28BE60DB9391054A7F09D5F47D4D3770
    for m, e in ((1 << 23, -23), (0xFFFFFF, -24), (0xABCDEF, -40), (0x800001, -60), (12345678, -22), (1, -149), (0xC90FDB, -21)):
        F = turn_fraction(m, e)
        for pos in (0, 1, -1, 7, 12345, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31):
            got = Fraction((pos * F) % 2 ** 64, 2 ** 64)
            want = Fraction(pos) * m * Fraction(2) ** e / two_pi
            off = (got - want) % 1
            assert min(off, 1 - off) <= Fraction(1, 2 ** 33)
