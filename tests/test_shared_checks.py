"""Refusals of the shared-prefix plan and attention, in the binding and at the C entries.  No GPU."""
import ctypes

import pytest
import torch

from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
from tests.test_binding_checks import _StubLib

H16, I32 = torch.float16, torch.int32


@pytest.fixture
def stub(monkeypatch):
    """The binding on host tensors, with entry points that only record the call."""
    lib = _StubLib()
    monkeypatch.setattr(LT, "load", lambda path=None: lib)
    monkeypatch.setattr(LT, "_device", lambda: -1)  # where host tensors are
    monkeypatch.setattr(LT, "_raw_stream", lambda stream, dev: 0)
    return lib


def plan(**over):
    a = dict(page_table=torch.zeros(4, 3, dtype=I32), ctx_len=torch.zeros(4, dtype=I32),
             group_start=torch.zeros(3, dtype=I32), N=3, Hq=4, Hkv=2, D=128, num_pages=5,
             shared_pages=torch.zeros(2, dtype=I32), plan=torch.zeros(256, dtype=torch.uint8),
             status=torch.zeros(1, dtype=I32))
    a.update(over)
    LT.lucetree_shared_plan(**a)


def attn(**over):
    B, N, Hq, Hkv, D, P = 2, 3, 4, 2, 128, 5
    a = dict(q=torch.zeros(B, N, Hq, D, dtype=H16), k_pool=torch.zeros(P, Hkv, 64, D, dtype=H16),
             v_pool=torch.zeros(P, Hkv, 64, D, dtype=H16), page_table=torch.zeros(B, 2, dtype=I32),
             ctx_len=torch.zeros(B, dtype=I32), k_tree=torch.zeros(B, N, Hkv, D, dtype=H16),
             v_tree=torch.zeros(B, N, Hkv, D, dtype=H16), anc_mask=torch.zeros(B, N, dtype=torch.int64), groups=1,
             plan=torch.zeros(256, dtype=torch.uint8), out=torch.zeros(B, N, Hq, D, dtype=H16),
             status=torch.zeros(1, dtype=I32), workspace=torch.zeros(256, dtype=torch.uint8))
    a.update(over)
    LT.lucetree_verify_attn_shared(**a)


def test_accepts(stub):
    plan()
    attn()
    attn(out=torch.zeros(2, 3, 4, 128), lse=torch.zeros(2, 3, 4))
    assert stub.calls == ["lucetree_shared_plan"] + ["lucetree_verify_attn_shared"] * 2


@pytest.mark.parametrize("go,bad", [
    (plan, dict(page_table=torch.zeros(4, 3, dtype=torch.int64))), (plan, dict(ctx_len=torch.zeros(3, dtype=I32))),
    (plan, dict(group_start=torch.zeros(3))), (plan, dict(shared_pages=torch.zeros(3, dtype=I32))), (plan, dict(N=0)),
    (plan, dict(num_pages=0)), (plan, dict(num_pages=1 << 31)), (plan, dict(plan=None)), (plan, dict(status=None)),
    (plan, dict(page_table=torch.zeros(3, 4, dtype=I32).T)),
    (attn, dict(out=torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16))), (attn, dict(out=torch.zeros(2, 3, 4, 64))),
    (attn, dict(groups=0)), (attn, dict(groups=1 << 31)), (attn, dict(plan=None)), (attn, dict(lse=torch.zeros(2, 3, 3))),
    (attn, dict(anc_mask=torch.zeros(2, 3, dtype=I32))), (attn, dict(k_tree=torch.zeros(2, 3, 2, 128))),
    (attn, dict(page_table=torch.zeros(1, 2, dtype=I32))), (attn, dict(workspace=None)),
])
def test_refuses(stub, go, bad):
    with pytest.raises(LT.LucetreeError):
        go(**bad)
    assert stub.calls == []


@pytest.mark.parametrize("go", [plan, attn])
def test_refuses_tensors_of_another_device(stub, monkeypatch, go):
    monkeypatch.setattr(LT, "_device", lambda: 0)
    with pytest.raises(LT.LucetreeError, match="cuda:0"):
        go()
    assert stub.calls == []


MB = 1 << 20  # addresses below are never dereferenced: every call is refused first


def test_sizes():
    lib, n = LT.load(), ctypes.c_size_t(0)
    for f in (lib.lucetree_shared_plan_bytes, lib.lucetree_verify_attn_shared_workspace):
        assert f(4, 3, 4, 2, 128, 2, ctypes.byref(n)) == 0 and n.value > 0
        assert f(4, 3, 4, 2, 128, 2, None) == 1
        for bad in ((0, 3, 4, 2, 128, 1), (4, 0, 4, 2, 128, 1), (4, 3, 4, 2, 128, 0), (4, 3, 4, 2, 128, 5), (4, 3, 0, 2, 128, 1)):
            assert f(*bad, ctypes.byref(n)) == 1, bad
        for bad in ((4, 65, 4, 2, 128, 1), (4, 3, 5, 2, 128, 1), (4, 3, 4, 2, 64, 1), (4, 3, 129, 1, 128, 1),
                    (1 << 26, 3, 16, 1, 128, 1), (1 << 21, 1, 2, 2, 128, 1)):
            assert f(*bad, ctypes.byref(n)) == 2, bad


def test_plan_entry_refuses_before_any_launch():
    lib = LT.load()
    ok = dict(B=4, N=3, Hq=4, Hkv=2, D=128, page_table=MB, max_pages_per_seq=8, num_pages=5, ctx_len=2 * MB, groups=2,
              group_start=3 * MB, shared_pages=4 * MB, plan=8 * MB, plan_bytes=4 * MB, status=5 * MB)

    def rc(**bad):
        return lib.lucetree_shared_plan(ctypes.byref(LT.SharedPlanArgs(**{**ok, **bad})), None)

    assert lib.lucetree_shared_plan(None, None) == 1
    for bad in (dict(B=0), dict(groups=0), dict(groups=5), dict(page_table=None), dict(ctx_len=None), dict(group_start=None),
                dict(shared_pages=None), dict(plan=None), dict(status=None), dict(max_pages_per_seq=0), dict(num_pages=0),
                dict(page_table=8 * MB), dict(ctx_len=8 * MB), dict(group_start=8 * MB + 64), dict(shared_pages=8 * MB),
                dict(shared_pages=2 * MB), dict(shared_pages=3 * MB + 8)):
        assert rc(**bad) == 1, bad
    for bad in (dict(N=65), dict(D=64), dict(Hq=5), dict(max_pages_per_seq=0x7fffffff)):
        assert rc(**bad) == 2, bad
    assert rc(plan_bytes=100) == 3 and rc(plan=8 * MB + 16) == 3


def test_attention_entry_refuses_before_any_launch():
    lib = LT.load()
    ok = dict(dtype=LT.LUCETREE_BF16, B=4, N=4, Hq=4, Hkv=2, D=128, page_size=64, scale=1.0, q=MB, k_pool=MB, v_pool=MB,
              num_pages=3, page_table=MB, max_pages_per_seq=2, ctx_len=MB, k_tree=MB, v_tree=MB, anc_mask=MB, status=MB)

    def rc(groups=2, plan=8 * MB, plan_bytes=4 * MB, out_dtype=LT.LUCETREE_F32, out=2 * MB, **attn):
        w = LT.SharedArgs()
        w.attn = LT.AttnArgs(**{**ok, **attn})
        w.groups, w.plan, w.plan_bytes, w.out_dtype, w.out = groups, plan, plan_bytes, out_dtype, out
        return lib.lucetree_verify_attn_shared(ctypes.byref(w), None, 0, None)

    assert lib.lucetree_verify_attn_shared(None, None, 0, None) == 1
    assert rc() == 3  # all fine but the workspace
    assert rc(plan_bytes=100) == 3 and rc(plan=8 * MB + 8) == 3
    for bad in (dict(groups=0), dict(groups=5), dict(plan=None), dict(out=None), dict(out=2 * MB + 4), dict(out=MB),
                dict(out=8 * MB), dict(q=None), dict(anc_mask=None), dict(num_pages=0), dict(scale=float("nan"))):
        assert rc(**bad) == 1, bad
    for bad in (dict(out_dtype=LT.LUCETREE_F16), dict(out_dtype=7), dict(dtype=LT.LUCETREE_F32), dict(D=64), dict(N=65),
                dict(Hq=5)):
        assert rc(**bad) == 2, bad
