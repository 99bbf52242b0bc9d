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


def test_outputs_of_a_selection():
    ok = dict(dtype=2, batch=2, beams_in=4, beams_out=4, vocab=50, row_stride=50, logits=AT, cum=AT + 4096,
              finished=AT + 8192, eos=1, out_score=AT + 12288, out_token=AT + 16384, out_row=AT + 20480,
              out_finished=AT + 24576)
    outs = ("out_score", "out_token", "out_row", "out_finished")
    lib = LT.load()

    def rc(**change):
        a = LT.BeamArgs(**{**ok, **change})
        return lib.lucetree_beam_select(ctypes.byref(a), 1 << 24, 1 << 20, None)

    for at in (-28, 0, 28):                            # (32 bytes each)
        for name in outs:
            for other in ("cum", "finished", *outs):
                if name != other and (name, other, at) not in (("out_score", "cum", 0), ("out_finished", "finished", 0)):
                    assert rc(**{name: ok[other] + at}) == 1, (name, other, at)
