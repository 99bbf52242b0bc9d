"""bf16 values too small for fp16's normal range: off by at most half of its smallest step, 2^-25,
where the product runs on fp16, and not at all with a bf16 output."""
import pytest
import torch

from tests.test_gpu_attention_steep_full import run
from tests.test_gpu_attention_window import P_STEP, call, make, reference



def small(window, size):
    s = make((700, 65, 0, 300), 5, 8, 2, 128, "bf16", window, 0, "chain", seed=51)
    for name in ("v_pool", "v_tree"):
        s[name] = (s[name].float() * size).bfloat16()
    return s


def test_which_values_are_exact():
    v = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[v.float() < 65536]
    off = (v.to(torch.float16).double() - v.double()).abs()
    assert (off[v.float() >= 2.0 ** -17] == 0).all() and off.max() <= 2.0 ** -25 and off[v.float() < 2.0 ** -17].max() > 0


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-5, 1e-6, 1e-8])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_windowed(cuda_dev, size, out):
    s = small(200, size)
    got, _, status = call(s, out)
    ref, _, bound, _ = reference(s, None, P_STEP[out])
    # (the weights sum to 1: a convex sum of errors of at most 2^-25, and bound's 2^-11 of each)
    extra = 2.0 ** -25 * (1 + 2.0 ** -10) if out == torch.float32 else (bound + ref.abs()) * 2.0 ** -8
    assert status == 0 and ((got.double() - ref).abs() <= bound + 2.0 ** -24 * ref.abs() + extra).all()


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1.0, 1e-5, 1e-8])
def test_full(cuda_dev, size):
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    s = small(1 << 20, size)
    got, _, status = run(s, LT.lucetree_verify_attn, LT.lucetree_verify_attn_workspace)
    ref, _, bound, _ = reference(s, None, P_STEP[torch.float32])
    assert status == 0
    assert ((got.double() - ref).abs() <= bound + 2.0 ** -24 * ref.abs() + 2.0 ** -25 * (1 + 2.0 ** -10)).all()
