"""Page-table calls at their largest sizes: refusals on the host, and counts next to 2^31."""
import ctypes

import pytest
import torch

from speculative_decoding_tree_ddtree_gb300 import lucetree as LT

AT = 1 << 20
TOP = 2 ** 31 - 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses stay off the GPU")
def test_refusals():
    lib = LT.load()
    ok = dict(table_in=AT, ctx_len=AT, rows=3, max_pages_per_seq=4, window=5, sinks=0, ref_in=AT, num_pages=9, table_out=AT,
              ref_out=AT, status=AT)
    for change in (dict(rows=TOP), dict(rows=TOP - 65534), dict(max_pages_per_seq=TOP), dict(max_pages_per_seq=TOP - 1023)):
        assert lib.lucetree_trim_pages(ctypes.byref(LT.TrimArgs(**{**ok, **change})), None) == 2, change
    far = 1 << 40
    ok = dict(table_in=far, ctx_in=2 * far, rows_in=3, src=3 * far, rows_out=3, max_pages_per_seq=1, reserve=2, ref_in=4 * far,
              num_pages=9, table_out=5 * far, ctx_out=6 * far, ref_out=4 * far, copy_src=7 * far, copy_dst=8 * far, status=AT)
    for change, want in ((dict(), 3), (dict(rows_in=TOP), 2), (dict(rows_out=TOP), 2), (dict(max_pages_per_seq=TOP), 2),
                         (dict(rows_in=1 << 30, rows_out=1 << 30), 2), (dict(rows_in=1 << 30, rows_out=(1 << 30) - 65536), 3),
                         (dict(rows_out=TOP // 64, reserve=4032), 3), (dict(rows_out=TOP // 64 + 1, reserve=4032), 2)):
        a = LT.ReorderArgs(**{**ok, **change})
        assert lib.lucetree_reorder_pages(ctypes.byref(a), None, 0, None) == want, change


@pytest.mark.gpu
def test_counts_of_as_many_pages_as_an_int_names(cuda_dev):
    i32 = dict(dtype=torch.int32, device="cuda")
    ref = torch.ones(TOP, **i32)
    ref2, st = torch.zeros(TOP, **i32), torch.zeros(1, **i32)
    table, ctx = torch.tensor([[TOP - 1, 5, 7]], **i32), torch.tensor([150], **i32)
    LT.lucetree_trim_pages(table, ctx, 1, 0, ref, table, ref2, st)
    assert int(st.item()) == 0 and table.tolist() == [[-1, -1, 7]]
    assert int(ref2[TOP - 1]) == 0 and int(ref2[5]) == 0
    ref2[[TOP - 1, 5]] = 1
    assert torch.equal(ref, ref2)
