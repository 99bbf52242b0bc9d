"""Values that are not finite in the tree: nodes that do not see them, such as the real nodes of
a padded tree, are as without them."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attention_window import P_STEP, call, make, reference

pytestmark = pytest.mark.gpu

SHAPES = {
    "whole":  ((400, 0, 65) * 12, 5, 4, 2, 128, 200),
    "split":  ((1000, 700, 930, 64) * 10, 4, 8, 4, 128, 900),
    "split-256": ((900, 500) * 14, 3, 12, 4, 256, 850),
    "wide":   ((700, 40) * 6, 22, 24, 4, 256, 600),
    "small-window": ((300,) * 8, 40, 2, 1, 128, 5),   # deep nodes no longer see the first ones
    "all-nodes": ((500,) * 6, 64, 2, 2, 128, 300),
}


def sees(s, b, i, j):
    """Whether node i of sequence b sees node j."""
    path = s["paths"][b * s["q"].shape[1] + i]
    L = int(s["ctx_len"][b])
    return j in path and (L + path.index(j) < s["sinks"] or len(path) - 1 - path.index(j) < s["window"])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "same"), ("f16", "same")])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_nodes_that_do_not_see_them(cuda_dev, shape, dtype, out, value):
    ctx, N, Hq, Hkv, D, window = SHAPES[shape]
    s = make(ctx, N, Hq, Hkv, D, dtype, window, 4, "chain" if shape == "small-window" else "random", seed=41)
    rng = np.random.default_rng(5)
    bad = {b: int(rng.integers(0, N)) for b in range(0, len(ctx), 2)}
    out_dtype = torch.float32 if out == "f32" else s["q"].dtype
    ref, ref_lse, bound, lse_bound = reference(s, None, P_STEP[out_dtype])
    for n, (b, j) in enumerate(bad.items()):
        if n % 2:
            s["k_tree"][b, j, :, 3] = float("nan")
        s["v_tree"][b, j, :, [(7 * n) % D, D - 1]] = value
    got, lse, status = call(s, out_dtype)
    bound = bound + (0 if out_dtype == torch.float32 else torch.finfo(out_dtype).eps / 2) * (ref.abs() + bound)
    fine = torch.ones(len(ctx), N, dtype=torch.bool)
    for b, j in bad.items():
        for i in range(N):
            fine[b, i] = not sees(s, b, i, j)
    assert fine.any() and not fine.all()
    assert ((got[fine].double() - ref[fine]).abs() <= bound[fine] + 2.0 ** -24 * ref[fine].abs()).all()
    assert ((lse[fine].double() - ref_lse[fine]).abs() <= lse_bound[fine]).all()
    assert not torch.isfinite(got[~fine]).all(-1).any()
    assert status == 0x40                            # DEV_NONFINITE


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_nodes_that_nobody_sees(cuda_dev, dtype):
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    s = make((300, 900, 20), 9, 8, 2, 128, dtype, 200, 4, "chain", seed=43)
    ref, _, bound, _ = reference(s, None, P_STEP[s["q"].dtype])
    s["anc_mask"][:, 6:] = 0                         # the last three are padding
    s["k_tree"][:, 6:] = float("nan")
    s["v_tree"][:, 6:] = float("nan")
    got, lse, status = call(s, s["q"].dtype)
    assert status == LT.DEV_BAD_NODE
    bound = bound + torch.finfo(got.dtype).eps / 2 * (ref.abs() + bound)
    assert ((got[:, :6].double() - ref[:, :6]).abs() <= bound[:, :6]).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_values_beyond_fp16(cuda_dev, out):
    """bf16 V from 65,536 on: the rows that see it are flagged where V is converted, the others stay."""
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    s = make((300, 900), 6, 8, 2, 128, "bf16", 200, 4, "chain", seed=44)
    s["v_tree"][0, 4, 1, 5] = 1e5
    ref, _, bound, _ = reference(s, None, P_STEP[out])
    got, _, status = call(s, out)
    bound = bound + (0 if out == torch.float32 else 2.0 ** -8) * (ref.abs() + bound) + 2.0 ** -24 * ref.abs()
    ok = torch.ones(got.shape[:3], dtype=torch.bool)
    if out == torch.float32:
        ok[0, 4:, 4:] = False                        # descendants, heads of KV head 1
        assert not torch.isfinite(got[~ok]).all(-1).any()
    assert status == (LT.DEV_NONFINITE if out == torch.float32 else 0)
    assert ((got[ok].double() - ref[ok]).abs() <= bound[ok]).all()
