"""Layouts that mt_rope_append refuses because two of the rows that it writes
would share elements, and those it takes (no device needed)."""
import pytest

from test_paged_host import A, ALIAS, OK, SHAPE, batch, cache, mt, rope  # noqa: F401  (mt: a fixture)

NHD = dict(page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64)


@pytest.mark.parametrize("kw", [
    dict(NHD, token_stride=64), dict(NHD, head_stride=128), dict(NHD, page_stride=64), dict(NHD, page_stride=16 * 2 * 64 - 8),
    dict(NHD, page_stride=15 * 128 + 64), dict(page_stride=2048, token_stride=64, head_stride=15 * 64),
    dict(page_stride=2048, token_stride=64, head_stride=64), dict(page_stride=128, token_stride=128, head_stride=64),
    dict(page_stride=128, token_stride=1024, head_stride=64)], ids=str)  # 10 pages of 128 between tokens 1024 apart
def test_rows_that_share_elements(mt, kw):  # noqa: F811
    assert rope(mt, c=cache(mt, **kw), b=batch(mt, T=0)) == SHAPE


@pytest.mark.parametrize("kw", [
    NHD, dict(page_stride=2048, token_stride=64, head_stride=16 * 64),                     # heads outside, tokens inside
    dict(NHD, page_stride=2 * 2048, v=A(0) + 2 * 2048),                                    # K and V of a page side by side
    dict(page_stride=2 * 2048, token_stride=256, head_stride=64, v=A(0) + 2 * 128),        # of a token
    dict(page_stride=2 * 2048, token_stride=256, head_stride=128, v=A(0) + 2 * 64),        # of a head
    dict(page_stride=2 * 2048, token_stride=256, head_stride=128, k=A(0) + 2 * 64, v=A(0)),
    dict(page_stride=128, token_stride=10 * 128, head_stride=64),                          # a page's tokens far apart
    dict(page_stride=64, token_stride=10 * 64, head_stride=160 * 64),                      # heads outermost
    dict(page_stride=0, token_stride=0, head_stride=0, num_pages=1, page_size=1, kv_heads=1),
    dict(NHD, head_stride=8, kv_heads=1), dict(NHD, num_pages=1, page_stride=8)], ids=str)
def test_rows_that_do_not(mt, kw):  # noqa: F811
    assert rope(mt, c=cache(mt, **kw), b=batch(mt, T=0)) == OK


@pytest.mark.parametrize("kw", [
    dict(NHD, v=A(0)), dict(NHD, v=A(0) + 2 * 56), dict(NHD, v=A(0) + 2 * 128), dict(NHD, v=A(0) + 2 * 2048 * 9),
    dict(NHD, k=A(0) + 2 * 2048 * 9 + 2 * 8, v=A(0)), dict(NHD, page_stride=2 * 2048, v=A(0) + 2 * (2048 - 64)),
    dict(NHD, page_stride=2 * 2048, v=A(0) + 2 * 4096 * 3), dict(NHD, head_stride=8, kv_heads=1, v=A(0) + 2 * 56)], ids=str)
def test_rows_of_v_in_rows_of_k(mt, kw):  # noqa: F811
    assert rope(mt, c=cache(mt, **kw), b=batch(mt, T=0)) == ALIAS


def test_against_sets_of_elements(mt):  # noqa: F811
    # every combination of a few strides and offsets, against the elements themselves
    d, n_page, n_tok, n_head = 16, 3, 2, 2
    rows = [(p, t, h) for p in range(n_page) for t in range(n_tok) for h in range(n_head)]
    seen = set()
    for ps in (16, 32, 48, 64, 96, 128):
        for ts in (16, 32, 48, 96):
            for hs in (16, 24, 32, 64, 192):
                at = [p * ps + t * ts + h * hs for p, t, h in rows]
                apart = len({a + e for a in at for e in range(d)}) == len(at) * d
                for off in (-32, 0, 8, 16, 24, 32, 64, 200, 640):
                    got = rope(mt, c=cache(mt, page_stride=ps, token_stride=ts, head_stride=hs, num_pages=n_page, page_size=n_tok,
                                           kv_heads=n_head, head_dim=d, v=A(0) + 2 * off), b=batch(mt, T=0), rot=16)
                    k = {a + e for a in at for e in range(d)}
                    v = {a + off + e for a in at for e in range(d)}
                    if got == SHAPE:
                        # strides that do not nest are refused, even where the sizes happen to keep the rows apart
                        (s0, n0), (s1, n1), (s2, _) = sorted([(ps, n_page), (ts, n_tok), (hs, n_head)])
                        assert not apart or s1 < s0 * (n0 - 1) + d or s2 < s1 * (n1 - 1) + s0 * (n0 - 1) + d
                    else:
                        assert apart and got == (ALIAS if k & v else OK)
                    seen.add((got, apart))
    assert {(SHAPE, False), (OK, True), (ALIAS, True)} <= seen
