"""Buffers that the C entries refuse because they overlap.  Every call below is refused, so
the addresses are never used; without a GPU nothing could be launched either."""
import ctypes

import pytest
import torch

from speculative_decoding_tree_ddtree_gb300 import lucetree as LT

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses stay off the GPU")
AT = 1 << 20


def test_source_rows_under_an_output():
    ok = dict(table_in=AT, ctx_in=AT + 4096, rows_in=3, src=AT + 8192, rows_out=3, max_pages_per_seq=4, reserve=2,
              ref_in=AT + 12288, num_pages=9, table_out=AT + 16384, ctx_out=AT + 20480, ref_out=AT + 12288,
              copy_src=AT + 24576, copy_dst=AT + 28672, status=AT + 32768)

    def rc(**change):
        return LT.load().lucetree_reorder_pages(ctypes.byref(LT.ReorderArgs(**{**ok, **change})), None, 0, None)

    assert rc() == 3                                   # all fine but the workspace
    for at in (AT + 16384, AT + 16384 + 44, AT + 16384 - 8, AT + 12288, AT + 12288 + 32, AT + 12288 - 8):
        assert rc(src=at) == 1, at
    for at in (AT + 16384 + 48, AT + 16384 - 12, AT + 12288 + 36, AT + 12288 - 12):
        assert rc(src=at) == 3, at
