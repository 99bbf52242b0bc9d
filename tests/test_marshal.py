"""The binding's tensor check in C gives the address, or the error, of the one in Python."""

import pytest
import torch

from speculative_decoding_tree_ddtree_gb300 import lucetree as LT

BASE = torch.zeros(4, 6, dtype=torch.int32)

# tensor, kind, device, sizes
GOOD = [
    (BASE, "I32", -1, (4, 6)),
    (BASE, "W32", -1, (4, 6)),
    (BASE, "ANY", -1, ()),
    (BASE[1:3], "I32", -1, (2, 6)),
    (BASE[:, :1].contiguous(), "I32", -1, (4, 1)),
    (torch.zeros(0, dtype=torch.int32), "I32", -1, (0,)),
    (torch.zeros(3), "F32", -1, (3,)),
    (torch.zeros(2, 2, dtype=torch.float16), "F16", -1, (2, 2)),
    (torch.zeros(2, 2, dtype=torch.bfloat16), "BF16", -1, (2, 2)),
    (torch.zeros(5, dtype=torch.int64), "W64", -1, (5,)),
    (torch.zeros(7, dtype=torch.uint8), "ANY", -1, ()),
    (torch.nn.Parameter(torch.zeros(3)), "F32", -1, (3,)),
]
BAD = [
    (None, "I32", -1, (4, 6)),
    (BASE, "F32", -1, (4, 6)),
    (BASE, "W64", -1, (4, 6)),
    (BASE, "I32", -1, (4, 5)),
    (BASE, "I32", -1, (24,)),
    (BASE, "I32", -1, (4, 6, 1)),
    (BASE, "I32", 0, (4, 6)),
    (BASE.t(), "I32", -1, (6, 4)),
    (BASE[:, ::2], "I32", -1, (4, 3)),
    (BASE[:, :1].expand(4, 6), "I32", -1, (4, 6)),
    (torch.zeros(2, 2), "F16", -1, (2, 2)),
    (torch.zeros(2, 2, dtype=torch.float16), "BF16", -1, (2, 2)),
    (torch.zeros(0, dtype=torch.uint8), "ANY", -1, ()),
    (torch.zeros(3, device="meta"), "F32", 0, (3,)),
]


@pytest.fixture(scope="module")
def fast():
    if LT._arg is LT._arg_slow:
        pytest.skip("the compiled check was not built here")
    return LT._arg


def kind_of(name):
    return getattr(LT, "_K_" + name)


@pytest.mark.parametrize("i", range(len(GOOD)))
def test_addresses_agree(fast, i):
    t, kind, dev, sizes = GOOD[i]
    want = LT._arg_slow(t, "x", kind_of(kind), dev, *sizes)
    assert fast(t, "x", kind_of(kind), dev, *sizes) == want == t.data_ptr()


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals_agree(fast, i):
    t, kind, dev, sizes = BAD[i]
    with pytest.raises(LT.LucetreeError) as slow:
        LT._arg_slow(t, "x", kind_of(kind), dev, *sizes)
    with pytest.raises(LT.LucetreeError) as quick:
        fast(t, "x", kind_of(kind), dev, *sizes)
    assert str(quick.value) == str(slow.value) and "x" in str(quick.value)


@pytest.mark.parametrize("args", [(), (BASE,), (BASE, "x"), (BASE, "x", 1)])
def test_too_few_arguments(fast, args):
    with pytest.raises(TypeError):
        fast(*args)


@pytest.mark.parametrize("obj", [3, "text", [1, 2], BASE.numpy()])
def test_not_a_tensor(fast, obj):
    with pytest.raises(Exception):
        fast(obj, "x", LT._K_I32, -1, 4, 6)


def test_kind_out_of_range(fast):
    with pytest.raises(IndexError):
        fast(BASE, "x", 99, -1, 4, 6)


def test_no_reference_is_kept(fast):
    import sys
    t = torch.zeros(3)
    before = sys.getrefcount(t)
    for _ in range(10):
        fast(t, "x", LT._K_F32, -1, 3)
        with pytest.raises(LT.LucetreeError):
            fast(t, "x", LT._K_I32, -1, 3)
    assert sys.getrefcount(t) == before


def test_python_path_serves_the_same_call(monkeypatch):
    """Without the compiled check the entries take the same tensors."""
    monkeypatch.setattr(LT, "_arg", LT._arg_slow)
    monkeypatch.setattr(LT, "_device", lambda: -1)
    monkeypatch.setattr(LT, "_raw_stream", lambda s, d: 0)
    seen = []

    class Lib:
        def lucetree_trim_pages(self, args, stream):
            seen.append(args)
            return 0

    monkeypatch.setattr(LT, "load", lambda path=None: Lib())
    table, ctx, ref = BASE[:2].clone(), torch.ones(2, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32)
    LT.lucetree_trim_pages(table, ctx, 8, 1, ref, table.clone(), ref.clone(), status)
    assert len(seen) == 1 and len(seen[0]) == LT._TRIM_ARGS.size
