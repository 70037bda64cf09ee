"""Sizes at which the prompt-side operators' counts would leave an int: refused on the host."""
import pytest


@pytest.fixture(scope="module")
def pm():
    import bitplane_mixed_precision_b200 as pm
    return pm


A = 1 << 20  # an address with every alignment that a call asks for; refused calls never follow it


def code(pm, rows, E, N, gather):
    with pytest.raises(pm.PmoeError) as ei:
        pm.grouped_matmul(pm.make_dense(pm.BF16, A, None, E, N, 64),
                          pm.make_rows(pm.BF16, A, None, 1000 if gather else rows, A if gather else None), A, rows,
                          pm.F32, A)
    return ei.value.code


@pytest.mark.parametrize("gather", [False, True])
def test_tiles_that_a_step_past_the_last_would_bring_out_of_an_int(pm, gather):
    """If every expert claimed every row there would be rows / 128 * E * N / 256 tiles: within 148 of 2^31 a step past
    the last one wraps. Addresses that are no device memory are what stops the calls below that."""
    rows = 2113665 * 128  # 1016 experts: 2^31 - 8 tiles
    assert code(pm, rows, 1016, 256, gather) == 7
    assert code(pm, rows + 128, 1016, 256, gather) == 7
    assert code(pm, rows - 128, 1016, 256, gather) in (1, 2)  # 2^31 - 1024


@pytest.mark.parametrize("gather", [False, True])
def test_rows_whose_last_tile_would_leave_an_int(pm, gather):
    assert code(pm, 2 ** 31 - 1, 1, 8, gather) == 7
    assert code(pm, 2 ** 31 - 128, 1, 8, gather) == 7
    assert code(pm, 2 ** 31 - 129, 1, 8, gather) in (1, 2)


def test_widths_of_the_norm(pm):
    """Rows of 8-bit codes come in 128 columns; bf16 rows alone in 8, as bf16 matrices take them."""
    for H, outs, want in ((136, (A, A, A), 1), (136, (A, A, None), 1), (132, (None, None, A), 1), (4, (None, None, A), 1),
                          (136, (None, None, A), None), (8, (None, None, A), None)):
        if want is None:
            pm.residual_norm_q8(A, A, A, 0.0, 0, H, *outs)  # no rows: nothing to do
        else:
            with pytest.raises(pm.PmoeError) as ei:
                pm.residual_norm_q8(A, A, A, 0.0, 0, H, *outs)
            assert ei.value.code == want
