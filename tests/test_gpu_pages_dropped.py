"""Reordering with lengths near the end of the table."""
import numpy as np
import pytest

from tests.test_gpu_pages import PAGE, _lt, draw_pool, ref_reorder, run_reorder

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,P", [(4, 6), (30, 300)])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_full_row_that_ends_flags_nothing(cuda_dev, rows, P, in_place):
    rng = np.random.default_rng(rows)
    L = rng.integers(0, P * PAGE - 30, size=rows)
    L[1], L[2] = P * PAGE, P * PAGE - 5              # no room for the reserve
    table, L, ref = draw_pool(rng, rows, P, 4 * rows, L)
    src = rng.integers(-1, rows, size=rows)
    src[(src == 1) | (src == 2)] = 0
    *got, status = run_reorder(table, L, ref, src, 30, in_place)
    *want, short = ref_reorder(table, L, ref, src, 30)
    assert not short and status == 0
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("rows,P", [(4, 6), (30, 300)])
def test_a_full_row_that_goes_on_is_mapped_as_far_as_the_table_goes(cuda_dev, rows, P):
    rng = np.random.default_rng(rows)
    L = rng.integers(0, P * PAGE - 200, size=rows)
    L[1], L[2] = P * PAGE, P * PAGE - 70
    table, L, ref = draw_pool(rng, rows, P, 9 * rows, L)
    src = np.concatenate([[2, 1, 1, 2], rng.integers(-1, rows, size=rows)])
    *got, status = run_reorder(table, L, ref, src, 150)
    *want, short = ref_reorder(table, L, ref, src, 150)
    assert not short and status == _lt().DEV_BAD_CTX
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
