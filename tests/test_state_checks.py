"""Refusals of the beam selection, the page-table calls and the copies, in the
binding and at the C entries.  No GPU."""
import ctypes

import pytest
import torch

from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
from tests.test_binding_checks import _StubLib


@pytest.fixture
def stub(monkeypatch):
    """The binding on host tensors, with entry points that only record the call."""
    lib = _StubLib()
    monkeypatch.setattr(LT, "load", lambda path=None: lib)
    monkeypatch.setattr(LT, "_device", lambda: -1)  # where host tensors are
    monkeypatch.setattr(LT, "_raw_stream", lambda stream, dev: 0)
    return lib

I32 = torch.int32
FAKE = 1 << 20  # never dereferenced: every call below is refused first


def i32(*shape):
    return torch.zeros(*shape, dtype=I32)


def beam(**over):
    a = dict(logits=torch.zeros(2, 3, 50), cum=torch.zeros(2, 3), finished=i32(2, 3), eos=4, out_score=torch.zeros(2, 5),
             out_token=i32(2, 5), out_row=i32(2, 5), out_finished=i32(2, 5), workspace=torch.zeros(256, dtype=torch.uint8))
    a.update(over)
    LT.lucetree_beam_select(**a)


def reorder(**over):
    a = dict(table_in=i32(3, 4), ctx_in=i32(3), src=i32(5), reserve=2, ref_in=i32(9), table_out=i32(5, 4), ctx_out=i32(5),
             ref_out=i32(9), copy_src=i32(5), copy_dst=i32(5), status=i32(1), workspace=torch.zeros(256, dtype=torch.uint8))
    a.update(over)
    LT.lucetree_reorder_pages(**a)


def trim(**over):
    a = dict(table_in=i32(3, 4), ctx_len=i32(3), window=5, sinks=0, ref_in=i32(9), table_out=i32(3, 4), ref_out=i32(9),
             status=i32(1))
    a.update(over)
    LT.lucetree_trim_pages(**a)


def compact(**over):
    a = dict(table_in=i32(3, 4), ref_in=i32(9), table_out=i32(3, 4), ref_out=i32(9), copy_src=i32(4), copy_dst=i32(4),
             copy_n=i32(1), live=i32(1), status=i32(1), workspace=torch.zeros(256, dtype=torch.uint8))
    a.update(over)
    LT.lucetree_compact_pages(**a)


def copy(**over):
    a = dict(src=i32(4), dst=i32(4), k_pool=torch.zeros(9, 2, 64, 8), v_pool=torch.zeros(9, 2, 64, 4), status=i32(1),
             count=i32(1))
    a.update(over)
    LT.lucetree_copy_pages(**a)


def states(**over):
    a = dict(state_in=torch.zeros(3, 2, 8), src=i32(4), state_out=torch.zeros(4, 2, 8), status=i32(1))
    a.update(over)
    LT.lucetree_reorder_states(**a)


@pytest.mark.parametrize("go", [beam, reorder, trim, compact, copy, states])
def test_accepts(stub, go):
    go()
    assert len(stub.calls) == 1


def test_accepts_what_is_optional(stub):
    beam(finished=None, out_finished=None)
    beam(logits=torch.zeros(2, 3, 64)[:, :, :50])
    beam(logits=torch.zeros(2, 3, 50, dtype=torch.bfloat16), eos=-1)
    beam(logits=torch.zeros(2, 9, 50)[:, :1], cum=torch.zeros(2, 1), finished=None)  # one beam: rows any distance apart
    copy(v_pool=None, count=None)
    assert len(stub.calls) == 5


@pytest.mark.parametrize("go,bad", [
    (beam, dict(logits=torch.zeros(2, 3, 50, dtype=torch.float64))),
    (beam, dict(logits=torch.zeros(2, 50, 3).transpose(1, 2))),
    (beam, dict(logits=torch.zeros(2, 1, 50).expand(2, 3, 50))),
    (beam, dict(logits=torch.zeros(2, 4, 50)[:, :3])),
    (beam, dict(cum=torch.zeros(2, 3, dtype=torch.float64))), (beam, dict(cum=torch.zeros(2, 2))),
    (beam, dict(finished=torch.zeros(2, 3, dtype=torch.bool))), (beam, dict(out_token=i32(2, 4))),
    (beam, dict(out_row=torch.zeros(2, 5, dtype=torch.int64))), (beam, dict(out_finished=i32(2, 4))),
    (beam, dict(eos=1 << 31)),
    (reorder, dict(table_out=i32(5, 3))), (reorder, dict(table_in=torch.zeros(3, 4, dtype=torch.int64))),
    (reorder, dict(ctx_in=i32(2))), (reorder, dict(ref_out=i32(8))), (reorder, dict(copy_src=i32(4))),
    (reorder, dict(reserve=-1)), (reorder, dict(reserve=1 << 32)), (reorder, dict(src=None)),
    (reorder, dict(table_in=i32(4, 3).T)),
    (trim, dict(window=0)), (trim, dict(sinks=-1)), (trim, dict(table_out=i32(3, 3))), (trim, dict(ref_out=i32(8))),
    (trim, dict(window=1 << 31)),
    (compact, dict(copy_src=i32(3))), (compact, dict(copy_n=i32(2))), (compact, dict(live=None)),
    (compact, dict(table_out=i32(2, 4))),
    (copy, dict(dst=i32(3))), (copy, dict(v_pool=torch.zeros(8, 2, 64, 4))), (copy, dict(k_pool=torch.zeros(9))),
    (copy, dict(count=i32(2))), (copy, dict(src=torch.zeros(4, dtype=torch.int64))),
    (states, dict(state_out=torch.zeros(4, 2, 7))), (states, dict(state_out=torch.zeros(3, 2, 8))),
    (states, dict(state_out=torch.zeros(4, 2, 8, dtype=torch.float16))), (states, dict(state_in=torch.zeros(3))),
    (states, dict(status=None)),
])
def test_refuses(stub, go, bad):
    with pytest.raises(LT.LucetreeError):
        go(**bad)
    assert stub.calls == []


@pytest.mark.parametrize("go", [beam, reorder, trim, compact, copy, states])
def test_refuses_tensors_of_another_device(stub, monkeypatch, go):
    monkeypatch.setattr(LT, "_device", lambda: 0)
    with pytest.raises(LT.LucetreeError, match="cuda:0"):
        go()
    assert stub.calls == []


def test_sizes_of_workspaces():
    n = ctypes.c_size_t(0)
    lib = LT.load()
    for args, want in (((0, 1, 1, 5), 1), ((1, 33, 1, 5), 2), ((1, 1, 33, 50), 2), ((1, 2, 11, 5), 1), ((9000, 8, 8, 99), 2),
                       ((1, 1, 1, 0), 1)):
        assert lib.lucetree_beam_select_workspace(*args, ctypes.byref(n)) == want, args
    assert lib.lucetree_reorder_pages_workspace(0, 1, 1, ctypes.byref(n)) == 1
    assert lib.lucetree_reorder_pages_workspace(1, 1, (1 << 30) + 1, ctypes.byref(n)) == 2
    assert lib.lucetree_compact_pages_workspace(0, ctypes.byref(n)) == 1
    assert lib.lucetree_compact_pages_workspace((1 << 30) + 1, ctypes.byref(n)) == 2
    assert LT.lucetree_reorder_pages_workspace(3, 5, 9) > 0 and LT.lucetree_compact_pages_workspace(9) > 0


@pytest.mark.parametrize("entry,kind,ok,cases", [
    ("lucetree_beam_select", LT.BeamArgs,
     dict(dtype=2, batch=2, beams_in=3, beams_out=4, vocab=50, row_stride=50, logits=FAKE, cum=FAKE, out_score=FAKE + 24,
          out_token=FAKE, out_row=FAKE),
     [(dict(), 3), (dict(out_score=FAKE), 1), (dict(out_score=FAKE + 20), 1), (dict(beams_out=3, out_score=FAKE), 3),
      (dict(beams_out=3, out_score=FAKE + 4), 1), (dict(finished=FAKE, out_finished=FAKE), 1),
      (dict(beams_out=3, out_score=FAKE, finished=FAKE, out_finished=FAKE), 3), (dict(dtype=3), 2), (dict(batch=0), 1), (dict(beams_in=40), 2), (dict(row_stride=49), 1),
      (dict(logits=None), 1), (dict(logits=FAKE + 2), 1), (dict(dtype=1, logits=FAKE + 1), 1), (dict(cum=None), 1),
      (dict(out_row=None), 1), (dict(vocab=1), 1)]),
    ("lucetree_reorder_pages", LT.ReorderArgs,
     dict(table_in=FAKE, ctx_in=FAKE + 4096, rows_in=3, src=FAKE + 8192, rows_out=3, max_pages_per_seq=4, reserve=2, ref_in=FAKE,
          num_pages=9, table_out=FAKE + 48, ctx_out=FAKE, ref_out=FAKE, copy_src=FAKE, copy_dst=FAKE, status=FAKE),
     [(dict(), 3), (dict(src=FAKE), 1), (dict(copy_src=FAKE + 8200), 1), (dict(table_out=FAKE + 44), 1), (dict(table_out=FAKE), 1), (dict(ctx_out=FAKE + 4104), 1),
      (dict(ref_out=FAKE + 4), 1), (dict(reserve=4033), 2), (dict(reserve=-1), 1), (dict(rows_in=0), 1),
      (dict(num_pages=0), 1), (dict(num_pages=(1 << 30) + 1), 2), (dict(src=None), 1), (dict(copy_dst=None), 1)]),
    ("lucetree_compact_pages", LT.CompactArgs,
     dict(table_in=FAKE, rows=3, max_pages_per_seq=4, ref_in=FAKE, num_pages=9, table_out=FAKE, ref_out=FAKE, copy_src=FAKE,
          copy_dst=FAKE, copy_n=FAKE, live=FAKE, status=FAKE),
     [(dict(), 3), (dict(table_out=FAKE + 4), 1), (dict(ref_out=FAKE + 8), 1), (dict(rows=0), 1), (dict(copy_n=None), 1),
      (dict(copy_src=None), 1), (dict(num_pages=1, copy_src=None, copy_dst=None), 3)]),
])
def test_c_entries_with_a_workspace(entry, kind, ok, cases):
    lib = LT.load()
    assert getattr(lib, entry)(None, None, 0, None) == 1
    for change, want in cases:
        a = kind(**{**ok, **change})
        assert getattr(lib, entry)(ctypes.byref(a), None, 0, None) == want, change


@pytest.mark.parametrize("entry,kind,ok,cases", [
    ("lucetree_trim_pages", LT.TrimArgs,
     dict(table_in=FAKE, ctx_len=FAKE, rows=3, max_pages_per_seq=4, window=5, sinks=0, ref_in=FAKE, num_pages=9,
          table_out=FAKE, ref_out=FAKE, status=FAKE),
     [(dict(window=0), 1), (dict(sinks=-1), 1), (dict(rows=0), 1), (dict(table_out=FAKE + 4), 1), (dict(ref_out=FAKE + 4), 1),
      (dict(status=None), 1), (dict(ctx_len=None), 1)]),
    ("lucetree_copy_pages", LT.CopyPagesArgs,
     dict(src=FAKE, dst=FAKE, n=3, k_pool=FAKE, v_pool=FAKE, k_page_bytes=32, v_page_bytes=16, num_pages=4, status=FAKE),
     [(dict(n=-1), 1), (dict(n=0, src=None), 0), (dict(k_page_bytes=24), 1), (dict(v_page_bytes=0), 1), (dict(k_pool=None), 1),
      (dict(k_pool=FAKE + 8), 1), (dict(v_pool=FAKE + 4), 1), (dict(num_pages=0), 1), (dict(dst=None), 1)]),
    ("lucetree_reorder_states", LT.ReorderStatesArgs,
     dict(state_in=FAKE, state_out=FAKE + 96, src=FAKE, rows_in=3, rows_out=2, row_bytes=32, status=FAKE),
     [(dict(state_out=FAKE + 80), 1), (dict(state_out=FAKE), 1), (dict(row_bytes=8), 1), (dict(row_bytes=40), 1),
      (dict(rows_in=0), 1), (dict(src=None), 1), (dict(state_in=FAKE + 4), 1)]),
])
def test_c_entries_without_a_workspace(entry, kind, ok, cases):
    lib = LT.load()
    assert getattr(lib, entry)(None, None) == 1
    for change, want in cases:
        a = kind(**{**ok, **change})
        assert getattr(lib, entry)(ctypes.byref(a), None) == want, change
