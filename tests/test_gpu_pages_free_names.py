"""Table entries that name a page without a holder: flagged, and never another sequence's data."""
import numpy as np
import pytest
import torch

from tests.test_gpu_pages import _dev, _lt, _new, _status

pytestmark = pytest.mark.gpu


def compact(table, ref, in_place):
    LT = _lt()
    t, f, st = _dev(table), _dev(ref), _status()
    n = len(ref)
    t2, f2 = (t, f) if in_place else (_new(*np.shape(table)), _new(n))
    cs, cd, cn, live = _new(n // 2), _new(n // 2), _new(1), _new(1)
    ws = torch.empty(LT.lucetree_compact_pages_workspace(n), dtype=torch.uint8, device="cuda")
    ws.fill_(0xEE)
    LT.lucetree_compact_pages(t, f, t2, f2, cs, cd, cn, live, st, ws)
    return t2.cpu().numpy(), f2.cpu().numpy(), int(cn.item()), int(live.item()), int(st.item())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cols", [8, 3000])          # one launch, several
@pytest.mark.parametrize("pages", [8, 9000])
def test_compaction(cuda_dev, in_place, cols, pages):
    # pages 0, 2 and `last` are held; 1 is free below the live count and `last` moves there
    last = pages - 1
    ref = np.zeros(pages, int)
    ref[[0, 2, last]] = 1, 2, 1
    table = np.full((2, cols), -1)
    table[0, :4] = 0, 2, 1, 3                        # 1 and 3 have no holder
    table[1, -2:] = 2, last
    want = table.copy()
    want[0, 2:4], want[1, -1] = -1, 1
    new = np.zeros(pages, int)
    new[:3] = 1, 1, 2
    got = compact(table, ref, in_place)
    assert np.array_equal(got[0], want) and np.array_equal(got[1], new)
    assert got[2:] == (1, 3, _lt().DEV_BAD_PAGE)
