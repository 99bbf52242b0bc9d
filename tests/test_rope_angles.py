"""The rotation's steps at the borders of what they take.  No GPU."""
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
