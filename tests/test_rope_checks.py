"""The rotation's steps against their formulas, and the refusals of the rotation and of the appends, in the binding
and at the C entries.  No GPU."""
import ctypes
import math

import pytest
import torch

from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
from tests.test_binding_checks import _StubLib

H16, I32, I64 = torch.float16, torch.int32, torch.int64


@pytest.fixture
def stub(monkeypatch):
    """The binding on host tensors, with entry points that only record the call."""
    lib = _StubLib()
    monkeypatch.setattr(LT, "load", lambda path=None: lib)
    monkeypatch.setattr(LT, "_device", lambda: -1)  # where host tensors are
    monkeypatch.setattr(LT, "_raw_stream", lambda stream, dev: 0)
    return lib


# ------------------------------------------------------------------ steps

def formula(r, base, kind, s, C, low, high):
    if kind == LT.LUCETREE_ROPE_NTK:
        base = base * s ** (r / (r - 2))
    out = []
    d = lambda n: r * math.log(C / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
    for i in range(r // 2):
        f = base ** (-2 * i / r)
        if kind == LT.LUCETREE_ROPE_LINEAR:
            f /= s
        if kind == LT.LUCETREE_ROPE_BANDS:
            w = min(max((C * f / (2 * math.pi) - low) / (high - low), 0), 1)
            f = w * f + (1 - w) * f / s
        if kind == LT.LUCETREE_ROPE_YARN:
            lo, hi = max(math.floor(d(high)), 0), min(math.ceil(d(low)), r - 1)
            w = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
            f = w * f / s + (1 - w) * f
        out.append(f)
    return out


@pytest.mark.parametrize("r", [2, 4, 20, 64, 256])
@pytest.mark.parametrize("kind", range(5))
@pytest.mark.parametrize("base", [10000.0, 1e6])
def test_steps_are_the_formulas_fractions_of_a_turn(r, kind, base):
    if kind == LT.LUCETREE_ROPE_NTK and r == 2:
        return
    s, C, low, high = 8.0, 8192.0, 1.0, 32.0
    steps, m = LT.lucetree_rope_steps(r, base, scaling=kind, factor=s, orig_ctx=C, low=low, high=high)
    want = formula(r, base, kind, s, C, low, high)
    assert steps.shape == (r // 2,) and steps.dtype == I64
    for got, f in zip(steps.tolist(), want):
        got = (got % (1 << 64)) / 2.0 ** 64
        # a few roundings of 2^-53 in the power, the products and the quotient by 2 pi, and the step's own to
        # a whole multiple of 2^-64
        assert abs(got - f / (2 * math.pi)) <= 2.0 ** -48 * f + 2.0 ** -65
    assert m == pytest.approx(0.1 * math.log(s) + 1 if kind == LT.LUCETREE_ROPE_YARN else 1.0, rel=1e-7)


def test_divisors_and_a_given_magnitude():
    div = [1.0, 2.0, 0.25, 10.0]
    a, _ = LT.lucetree_rope_steps(8, 10000.0)
    b, m = LT.lucetree_rope_steps(8, 10000.0, factors=div)
    assert m == 1.0
    for x, y, d in zip(a.tolist(), b.tolist(), div):
        assert abs((y % 2 ** 64) - (x % 2 ** 64) / d) <= 2 ** 17  # of 2^64
    assert LT.lucetree_rope_steps(8, 1e4, scaling=4, factor=4.0, orig_ctx=4096, low=1, high=32, magnitude=1.5)[1] == 1.5


@pytest.mark.parametrize("bad", [
    dict(rot_dims=3), dict(rot_dims=0), dict(rot_dims=1026), dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")),
    dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("nan")),
    dict(scaling=2, factor=2.0, rot_dims=2), dict(scaling=3, factor=2.0), dict(scaling=3, factor=2.0, orig_ctx=100, low=4, high=1),
    dict(scaling=4, factor=2.0, orig_ctx=100, low=0, high=1), dict(scaling=4, factor=2.0, orig_ctx=9, low=1, high=2, magnitude=-1),
    dict(factors=[1.0, 0.0, 1.0, 1.0]), dict(factors=[1.0, 1.0]),
], ids=str)
def test_steps_refuse(bad):
    with pytest.raises(LT.LucetreeError):
        LT.lucetree_rope_steps(**{**dict(rot_dims=8, base=10000.0), **bad})


# ------------------------------------------------------------------ rows of a projection

def qkv(lead, Hq, Hkv, D, dtype=H16):
    x = torch.zeros(*lead, (Hq + 2 * Hkv) * D, dtype=dtype)
    return tuple(t.unflatten(-1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], -1))


ROWS = [(*qkv((2, 3), 4, 2, 16), 128), (*qkv((1, 3), 4, 2, 16), 128), (*qkv((5,), 1, 1, 32), 96)]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: str(tuple(c[0].shape)))
def test_rows_agree_with_the_python_check(case):
    for t in case[:3]:
        want = (t.data_ptr(), case[3])
        assert LT._rows(t, "x", LT._K_F16, -1, *t.shape) == LT._rows_slow(t, "x", LT._K_F16, -1, *t.shape) == want
    t = case[0].contiguous()
    assert LT._rows(t, "x", LT._K_F16, -1, *t.shape) == (t.data_ptr(), t.shape[-1] * t.shape[-2])


@pytest.mark.parametrize("t", [
    torch.zeros(2, 3, 4, 16, dtype=H16).transpose(2, 3), torch.zeros(2, 4, 3, 16, dtype=H16).transpose(1, 2),
    torch.zeros(2, 3, 4, 32, dtype=H16)[..., ::2], torch.zeros(2, 5, 4, 16, dtype=H16)[:, :3],
    torch.zeros(1, 1, 4, 16, dtype=H16).expand(2, 3, 4, 16), torch.zeros(2, 3, 4, 16),
    torch.zeros(2, 3, 1, 16, dtype=H16).expand(2, 3, 4, 16), None,
], ids=lambda t: "none" if t is None else str(t.stride()))
def test_rows_refuse_alike(t):
    shape = (2, 3, 4, 16)
    if t is not None and t.shape != shape:
        shape = tuple(t.shape)
    errors = []
    for f in (LT._rows, LT._rows_slow):
        with pytest.raises(LT.LucetreeError) as e:
            f(t, "x", LT._K_F16, -1, *shape)
        errors.append(str(e.value))
    assert errors[0] == errors[1] and "x" in errors[0]


# ------------------------------------------------------------------ binding

def rope(**over):
    B, N, Hq, Hkv, D = 2, 3, 4, 2, 32
    q, k, v = qkv((B, N), Hq, Hkv, D)
    a = dict(q=q, k=k, v=v, steps=torch.zeros(8, dtype=I64), layout=0, q_out=torch.zeros(B, N, Hq, D, dtype=H16),
             k_out=torch.zeros(B, N, Hkv, D, dtype=H16), v_out=torch.zeros(B, N, Hkv, D, dtype=H16),
             status=torch.zeros(1, dtype=I32), ctx_len=torch.zeros(B, dtype=I32), anc_mask=torch.zeros(B, N, dtype=I64))
    a.update(over)
    LT.lucetree_rope(**a)


def append(**over):
    T, Hq, Hkv, D, B, P = 5, 4, 2, 32, 3, 7
    q, k, v = qkv((T,), Hq, Hkv, D)
    pool = lambda: torch.zeros(P, Hkv, 64, D, dtype=H16)  # noqa: E731
    a = dict(q=q, k=k, v=v, start=torch.zeros(B + 1, dtype=I32), page_table=torch.zeros(B, 2, dtype=I32),
             ctx_len_in=torch.zeros(B, dtype=I32), ctx_len_out=torch.zeros(B, dtype=I32), k_pool=pool(), v_pool=pool(),
             status=torch.zeros(1, dtype=I32), q_out=torch.zeros(T, Hq, D, dtype=H16), steps=torch.zeros(8, dtype=I64))
    a.update(over)
    LT.lucetree_append_kv(**a)


def codes(D):
    return torch.zeros(7, 2, 64, D, dtype=torch.uint8), torch.zeros(7, 2, 64, dtype=torch.uint8)


def test_accepts(stub):
    rope()
    rope(v=None, v_out=None)
    rope(ctx_len=None, anc_mask=None, positions=torch.zeros(2, 3, dtype=I32))
    append()
    append(q=None, q_out=None, steps=None)
    append(k=torch.zeros(0, 2, 32, dtype=H16), v=torch.zeros(0, 2, 32, dtype=H16), q=None, q_out=None)
    c, e = codes(32)
    append(k_pool=c, k_exp=e)
    append(v_pool=c, v_exp=e, v_format=LT.LUCETREE_V_INT8)
    append(v_pool=codes(16)[0], v_exp=e, v_format=LT.LUCETREE_V_INT4)
    assert stub.calls == ["lucetree_rope"] * 3 + ["lucetree_append_kv"] * 6


@pytest.mark.parametrize("go,bad", [
    (rope, dict(q=torch.zeros(2, 3, 4, 32))), (rope, dict(k=torch.zeros(2, 3, 2, 32, dtype=torch.bfloat16))),
    (rope, dict(v=None)), (rope, dict(v_out=None)), (rope, dict(ctx_len=None)), (rope, dict(anc_mask=None)),
    (rope, dict(positions=torch.zeros(2, 3, dtype=I32))), (rope, dict(steps=torch.zeros(8))),
    (rope, dict(steps=torch.zeros(2, 4, dtype=I64))), (rope, dict(q_out=torch.zeros(2, 3, 4, 16, dtype=H16))),
    (rope, dict(k_out=torch.zeros(2, 3, 4, 32, dtype=H16)[:, :, ::2])), (rope, dict(layout=-1)), (rope, dict(status=None)),
    (rope, dict(ctx_len=torch.zeros(2, dtype=I64))), (rope, dict(anc_mask=torch.zeros(2, 3, dtype=I32))),
    (append, dict(v=torch.zeros(4, 2, 32, dtype=H16))), (append, dict(start=torch.zeros(3, dtype=I32))),
    (append, dict(q=None)), (append, dict(q_out=None)), (append, dict(k_exp=codes(32)[1])),
    (append, dict(v_exp=codes(32)[1])), (append, dict(v_format=1)), (append, dict(v_format=3)),
    (append, dict(v_format=2, v_pool=codes(32)[0], v_exp=codes(32)[1])), (append, dict(ctx_len_out=torch.zeros(2, dtype=I32))),
    (append, dict(k_pool=torch.zeros(7, 2, 32, 32, dtype=H16))), (append, dict(q_out=torch.zeros(5, 4, 16, dtype=H16))),
    (append, dict(page_table=torch.zeros(3, 2, dtype=I64))), (append, dict(steps=torch.zeros(8))),
])
def test_refuses(stub, go, bad):
    with pytest.raises(LT.LucetreeError):
        go(**bad)
    assert stub.calls == []


@pytest.mark.parametrize("go", [rope, append])
def test_refuses_tensors_of_another_device(stub, monkeypatch, go):
    monkeypatch.setattr(LT, "_device", lambda: 0)
    with pytest.raises(LT.LucetreeError, match="cuda:0"):
        go()
    assert stub.calls == []


# ------------------------------------------------------------------ C entries

MB = 1 << 20  # addresses below are never dereferenced: every call is refused first


def test_rope_entry_refuses_before_any_launch():
    lib = LT.load()
    ok = dict(dtype=LT.LUCETREE_BF16, B=2, N=4, Hq=4, Hkv=2, D=128, q=MB, k=2 * MB, v=3 * MB, q_stride=1024, k_stride=1024,
              v_stride=1024, steps=4 * MB, rot_dims=128, layout=0, magnitude=1.0, ctx_len=5 * MB, anc_mask=6 * MB,
              positions=None, q_out=7 * MB, k_out=8 * MB, v_out=9 * MB, status=10 * MB)

    def rc(**bad):
        a = LT.RopeArgs(**{**ok, **bad})
        return lib.lucetree_rope(ctypes.byref(a), None)

    assert lib.lucetree_rope(None, None) == 1
    for bad in (dict(B=0), dict(N=0), dict(Hq=0), dict(Hkv=0), dict(q=None), dict(k=None), dict(steps=None),
                dict(status=None), dict(v=None), dict(v_out=None), dict(q_out=None), dict(rot_dims=130), dict(rot_dims=3),
                dict(rot_dims=0), dict(magnitude=float("inf")), dict(ctx_len=None), dict(anc_mask=None),
                dict(q_stride=511), dict(q_stride=516), dict(k_stride=255), dict(v_stride=0), dict(q=MB + 8),
                dict(k_out=8 * MB + 2), dict(q_out=MB), dict(q_out=MB + 512), dict(k_out=3 * MB), dict(v_out=7 * MB + 16),
                dict(k_out=7 * MB), dict(q_out=4 * MB + 16), dict(k_out=5 * MB), dict(v_out=6 * MB + 32),
                dict(v_out=6 * MB, positions=6 * MB + 16, ctx_len=None, anc_mask=None)):
        assert rc(**bad) == 1, bad
    for bad in (dict(dtype=LT.LUCETREE_F32), dict(D=120), dict(D=1040), dict(layout=2), dict(layout=-1), dict(N=65),
                dict(B=1 << 20, N=1 << 11, positions=MB)):
        assert rc(**bad) == 2, bad


def test_append_entry_refuses_before_any_launch():
    lib = LT.load()
    ok = dict(dtype=LT.LUCETREE_BF16, B=2, rows=9, Hq=4, Hkv=2, D=256, page_size=64, q=MB, k=2 * MB, v=3 * MB,
              q_stride=2048, k_stride=2048, v_stride=2048, start=4 * MB, steps=5 * MB, rot_dims=64, layout=1, magnitude=1.0,
              page_table=6 * MB, max_pages_per_seq=4, num_pages=3, ctx_len_in=7 * MB, ctx_len_out=8 * MB, k_format=0,
              v_format=0, k_pool=9 * MB, v_pool=10 * MB, k_exp=None, v_exp=None, q_out=11 * MB, status=12 * MB)

    def rc(**bad):
        a = LT.AppendArgs(**{**ok, **bad})
        return lib.lucetree_append_kv(ctypes.byref(a), None)

    assert lib.lucetree_append_kv(None, None) == 1
    for bad in (dict(B=0), dict(rows=-1), dict(Hkv=0), dict(num_pages=0), dict(max_pages_per_seq=0), dict(q=None),
                dict(q_out=None), dict(k=None), dict(v=None), dict(start=None), dict(page_table=None), dict(status=None),
                dict(ctx_len_in=None), dict(ctx_len_out=None), dict(ctx_len_out=7 * MB), dict(ctx_len_out=7 * MB + 4),
                dict(k_pool=None), dict(k_format=1), dict(v_format=1), dict(v_format=2), dict(rot_dims=258), dict(Hq=0),
                dict(magnitude=float("nan")), dict(q_stride=1016), dict(k_stride=2052), dict(v=3 * MB + 8), dict(q_out=MB),
                dict(v_pool=9 * MB), dict(k_pool=2 * MB), dict(k_format=1, k_exp=9 * MB), dict(v_pool=6 * MB), dict(q_out=5 * MB)):
        assert rc(**bad) == 1, bad
    for bad in (dict(dtype=LT.LUCETREE_F32), dict(page_size=16), dict(D=264), dict(layout=2), dict(k_format=2),
                dict(v_format=3), dict(k_format=1, k_exp=13 * MB, dtype=LT.LUCETREE_F16),
                dict(k_format=1, k_exp=13 * MB, D=128), dict(v_format=1, v_exp=13 * MB, D=128),
                dict(max_pages_per_seq=1 << 25), dict(rows=0x7fffff00)):
        assert rc(**bad) == 2, bad
