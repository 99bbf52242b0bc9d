"""Refusals of the windowed attention, in the binding and at the C entry, and
its packed arguments.  No GPU."""
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


def _call(**over):
    B, N, Hq, Hkv, D, P = 2, 3, 4, 2, 128, 5
    h = torch.float16
    a = dict(q=torch.zeros(B, N, Hq, D, dtype=h), k_pool=torch.zeros(P, Hkv, 64, D, dtype=h),
             v_pool=torch.zeros(P, Hkv, 64, D, dtype=h), page_table=torch.zeros(B, 2, dtype=torch.int32),
             ctx_len=torch.zeros(B, dtype=torch.int32), k_tree=torch.zeros(B, N, Hkv, D, dtype=h),
             v_tree=torch.zeros(B, N, Hkv, D, dtype=h), anc_mask=torch.zeros(B, N, dtype=torch.int64), window=7,
             sinks=0, out=torch.zeros(B, N, Hq, D, dtype=h), status=torch.zeros(1, dtype=torch.int32),
             workspace=torch.zeros(256, dtype=torch.uint8))
    a.update(over)
    LT.lucetree_verify_attn_win(**a)


def test_accepts_both_output_types(stub):
    _call()
    _call(out=torch.zeros(2, 3, 4, 128), lse=torch.zeros(2, 3, 4))
    assert stub.calls == ["lucetree_verify_attn_win"] * 2


@pytest.mark.parametrize("bad", [
    dict(window=0), dict(window=-1), dict(window=1 << 31), dict(window=(1 << 32) + 5), dict(sinks=-1),
    dict(sinks=1 << 31), dict(out=torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16)),
    dict(out=torch.zeros(2, 3, 4, 128, dtype=torch.float64)), dict(out=torch.zeros(2, 3, 4, 64)),
    dict(lse=torch.zeros(2, 3, 3)), dict(anc_mask=torch.zeros(2, 3, dtype=torch.int32)),
    dict(k_pool=torch.zeros(5, 64, 2, 128, dtype=torch.float16).transpose(1, 2)),
], ids=str)
def test_refuses(stub, bad):
    with pytest.raises(LT.LucetreeError):
        _call(**bad)
    assert stub.calls == []


def test_refuses_tensors_of_another_device(stub, monkeypatch):
    monkeypatch.setattr(LT, "_device", lambda: 0)
    with pytest.raises(LT.LucetreeError, match="cuda:0"):
        _call()
    assert stub.calls == []


def test_c_entry_refuses_before_any_launch():
    lib = LT.load()
    fake = 1 << 20  # never dereferenced
    ok = dict(dtype=LT.LUCETREE_BF16, B=1, N=4, Hq=4, Hkv=2, D=128, page_size=64, scale=1.0, q=fake, k_pool=fake,
              v_pool=fake, num_pages=3, page_table=fake, max_pages_per_seq=2, ctx_len=fake, k_tree=fake, v_tree=fake,
              anc_mask=fake, status=fake)

    def rc(window=5, sinks=0, out_dtype=LT.LUCETREE_F32, out=fake + 65536, **attn):
        w = LT.WinArgs()
        w.attn = LT.AttnArgs(**{**ok, **attn})
        w.window, w.sinks, w.out_dtype, w.out = window, sinks, out_dtype, out
        return lib.lucetree_verify_attn_win(ctypes.byref(w), None, 0, None)

    assert lib.lucetree_verify_attn_win(None, None, 0, None) == 1
    assert rc() == 3  # all fine but the workspace
    for bad in (dict(window=0), dict(sinks=-1), dict(out=None), dict(out=fake + 65536 + 4), dict(out=fake), dict(out=fake + 4080), dict(q=None), dict(anc_mask=None),
                dict(num_pages=0), dict(scale=float("inf"))):
        assert rc(**bad) == 1, bad
    for bad in (dict(out_dtype=LT.LUCETREE_F16), dict(out_dtype=7), dict(dtype=LT.LUCETREE_F32), dict(D=64),
                dict(N=65), dict(Hq=5)):
        assert rc(**bad) == 2, bad
