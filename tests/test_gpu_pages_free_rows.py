"""Reordering rows with entries that name a page without a holder: such a page may be handed to
another row in the same call, so the entry counts as missing."""
import numpy as np
import pytest

from tests.test_gpu_pages import _lt, run_reorder

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [4, 700])           # one launch, two
@pytest.mark.parametrize("in_place", [False, True])
def test_entries_of_free_pages(cuda_dev, cols, in_place):
    L = np.array([138, 128, 100, 70])
    table = np.full((4, cols), -1)
    table[0, :3], table[1, :2], table[2, :2], table[3, :2] = (0, 1, 2), (3, 4), (5, 6), (8, 9)  # 4, 6 and 9 are free
    ref = np.zeros(12, int)
    ref[[0, 1, 2, 3, 5, 8]] = 1
    src = np.array([0, 0, 1, 1, 3])                  # row 2 ends
    out, ctx, new, cs, cd, status = run_reorder(table, L, ref, src, 20, in_place)
    want = np.full((5, cols), -1)
    want[0, :3], want[1, :3], want[2, :3], want[3, :3], want[4, :2] = (0, 1, 2), (0, 1, 4), (3, -1, 6), (3, -1, 7), (8, 9)
    assert np.array_equal(out, want) and ctx.tolist() == [138, 138, 128, 128, 70]
    assert new.tolist() == [2, 2, 1, 2, 1, 0, 1, 1, 1, 1, 0, 0]
    assert cs.tolist() == [-1, 2, -1, -1, -1] and cd.tolist() == [-1, 4, -1, -1, -1]
    assert status == _lt().DEV_BAD_PAGE
