"""Where k and v may lie when mt_rope_append turns q in place (no device
needed: what is refused never reaches one)."""
import pytest

from test_paged_host import A, ALIAS, batch, mt, rope  # noqa: F401  (mt: a fixture)

# q: 5 rows of 4 heads of 64 (256 elements); k and v: 2 heads (128)


@pytest.mark.parametrize("kw", [
    dict(k=A(5)), dict(v=A(5)), dict(k=A(5) + 2 * 128), dict(v=A(5) + 2 * 64, v_stride=256),
    dict(q_stride=512, q_out_stride=512, k=A(5) + 2 * 192, k_stride=512),      # the last of q's columns
    dict(q_stride=512, q_out_stride=512, v=A(5) + 2 * 448, v_stride=512),      # the next row's first
    dict(q_stride=512, q_out_stride=512, k=A(5) - 2 * 64, k_stride=512),       # from before the rows
    dict(q_stride=512, q_out_stride=512, k=A(5) + 2 * 256, k_stride=768)], ids=str)
@pytest.mark.parametrize("T", [1, 5])
def test_columns_of_q(mt, kw, T):  # noqa: F811
    if T == 1 and kw.get("v") == A(5) + 2 * 448 or T == 1 and kw.get("k_stride") == 768:
        pytest.skip("one row: beside q")
    assert rope(mt, b=batch(mt, T=T), q_out=A(5), **kw) == ALIAS


@pytest.mark.parametrize("kw", [
    dict(q_stride=512, q_out_stride=512, k=A(5) + 2 * 256, k_stride=512, v=A(5) + 2 * 384, v_stride=512),
    dict(q_stride=512, q_out_stride=512, k=A(5) - 2 * 256, k_stride=512, v=A(5) - 2 * 128, v_stride=512),
    dict(q_stride=512, q_out_stride=512, k=A(5) + 2 * 384, k_stride=1024),     # of every second row
    dict(q_stride=520, q_out_stride=520, k=A(5) + 2 * 392, k_stride=520)], ids=str)
@pytest.mark.parametrize("T", [1, 5])
def test_columns_beside_q(mt, kw, T):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up: what is accepted must not run")
    assert rope(mt, b=batch(mt, T=T), q_out=A(5), **kw) == mt.MT_ERR_CUDA  # accepted, and there is no device
