"""The rotation's steps to their last place, and at the borders of what they take.  No GPU."""
import math
from decimal import Decimal as Dec, getcontext

import pytest

from speculative_decoding_tree_ddtree_gb300 import lucetree as LT


@pytest.mark.parametrize("bad", [dict(factors=[1.0, 1.0, 1e-309, 1.0]), dict(factors=[5e-324, 1.0, 1.0, 1.0]),
                                 dict(scaling=4, factor=2.0, orig_ctx=9, low=1, high=2, magnitude=1e39)], ids=str)
def test_angles_and_magnitudes_that_are_not_finite_are_refused(bad):
    with pytest.raises(LT.LucetreeError):
        LT.lucetree_rope_steps(**{**dict(rot_dims=8, base=10000.0), **bad})


def test_the_smallest_divisors_are_taken():
    steps, _ = LT.lucetree_rope_steps(4, 10000.0, factors=[2.0 ** -1022, 1e300])
    assert steps.tolist()[1] == 0


PI = Dec("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211707")


def exact(r, base, kind, s, C, low, high, div):
    """The angles' fractions of a turn, times 2^64, from the formulas in 90 decimal digits."""
    getcontext().prec = 90
    b, s, C, low, high = Dec(base), Dec(s), Dec(C), Dec(low), Dec(high)
    if kind == LT.LUCETREE_ROPE_NTK:
        b = b * (s.ln() * Dec(r) / Dec(r - 2)).exp()
    d = lambda n: r * math.log(float(C) / (2 * math.pi * float(n))) / (2 * math.log(base))  # noqa: E731
    out = []
    for i in range(r // 2):
        f = (Dec(-2 * i) / Dec(r) * b.ln()).exp()
        if kind == LT.LUCETREE_ROPE_LINEAR:
            f /= s
        if kind == LT.LUCETREE_ROPE_BANDS:
            w = min(max((C * f / (2 * PI) - low) / (high - low), Dec(0)), Dec(1))
            f = w * f + (1 - w) * f / s
        if kind == LT.LUCETREE_ROPE_YARN:
            lo, hi = max(math.floor(d(high)), 0), min(math.ceil(d(low)), r - 1)
            w = min(max(Dec(i - lo) / max(Dec(hi - lo), Dec(0.001)), Dec(0)), Dec(1))
            f = w * f / s + (1 - w) * f
        out.append(f / Dec(div[i]) / (2 * PI) % 1 * 2 ** 64)
    return out


@pytest.mark.parametrize("r", [2, 4, 20, 128, 256, 1024])
@pytest.mark.parametrize("kind", range(5))
@pytest.mark.parametrize("base", [1.5, 10000.0, 5e5, 1e300])
@pytest.mark.parametrize("divided", [False, True])
def test_steps_to_half_a_unit(r, kind, base, divided):
    """Sums of two doubles carry some 100 bits: what is rounded is off by far less than 2^-20 units for angles of up to
    16 turns."""
    if kind == LT.LUCETREE_ROPE_NTK and r == 2:
        return
    s, C, low, high = 7.3, 8192.0, 1.0, 32.0
    div = [0.01 + 0.37 * i for i in range(r // 2)] if divided else [1.0] * (r // 2)
    steps, _ = LT.lucetree_rope_steps(r, base, scaling=kind, factor=s, orig_ctx=C, low=low, high=high,
                                      factors=div if divided else None)
    for got, want in zip(steps.tolist(), exact(r, base, kind, s, C, low, high, div)):
        far = (Dec(got % 2 ** 64) - want) % 2 ** 64
        assert min(far, 2 ** 64 - far) <= Dec(0.5) + Dec(2) ** -20
