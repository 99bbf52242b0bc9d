"""Attention whose scores rise steeply from one key tile to the next, against the
formula in 64 bits: a later key far above all before it makes the kernels take the
sums so far back and start from a new shift."""
import pytest
import torch

from tests.test_gpu_attention_window import P_STEP, call, make, reference

pytestmark = pytest.mark.gpu

PAGE = 64


def raise_keys(s, positions, heights, nodes=()):
    """Queries of 1/2 throughout, and the keys at these positions of every sequence (and of
    these nodes) of one value each, so that their scores are about `heights` (nats)."""
    D = s["q"].shape[-1]
    s["q"] = torch.full_like(s["q"], 0.5)
    for b in range(len(s["ctx_len"])):
        L = int(s["ctx_len"][b])
        for p, h in zip(positions, heights):
            if p < L:
                s["k_pool"][int(s["page_table"][b, p // PAGE]), :, p % PAGE] = h / (0.5 * D ** 0.5)
    for i, h in nodes:
        s["k_tree"][:, i] = h / (0.5 * D ** 0.5)
    return s


def compare(s, out, lse, status, out_dtype, scale=None):
    ref, ref_lse, bound, lse_bound = reference(s, scale, P_STEP[out_dtype])
    assert status == 0
    assert torch.isfinite(out).all()
    bound = bound + (0 if out_dtype == torch.float32 else torch.finfo(out_dtype).eps / 2) * (ref.abs() + bound)
    assert ((out.double() - ref).abs() <= bound + 2.0 ** -24 * ref.abs()).all()
    assert ((lse.double() - ref_lse).abs() <= lse_bound).all()


# segments of several tiles: left whole, cut over CTAs, and one row group of three column chunks a warp
SHAPES = {
    "whole": ((400,) * 50, 3, 4, 2, 128, 200),
    "split": ((1000, 700, 930, 64) * 10, 2, 8, 4, 128, 900),
    "split-256": ((900, 500) * 14, 3, 12, 4, 256, 850),
    "wide": ((700,) * 13, 22, 24, 4, 256, 600),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "same"), ("f16", "same")])
@pytest.mark.parametrize("how", ["scale", "one", "stairs", "node"])
def test_windowed(cuda_dev, shape, dtype, out, how):
    ctx, N, Hq, Hkv, D, window = SHAPES[shape]
    s = make(ctx, N, Hq, Hkv, D, dtype, window, 4, "chain", seed=31)
    scale = None
    if how == "scale":
        scale = 20.0
    else:
        raise_keys(s, *{"one": ([351, 620], [95.0, 300.0]), "stairs": (range(210, 1000, 70), [100.0 * k for k in range(1, 13)]),
                        "node": ([], [], [(N - 1, 250.0)])}[how])
    out_dtype = torch.float32 if out == "f32" else s["q"].dtype
    compare(s, *call(s, out_dtype, scale=scale), out_dtype, scale)


@pytest.mark.parametrize("height", [60, 85, 88, 89, 90, 120, 180, 500])
def test_windowed_by_height(cuda_dev, height):
    s = make((800, 410) * 20, 2, 4, 4, 128, "f16", 700, 0, "chain", seed=height)
    raise_keys(s, [390], [height])
    compare(s, *call(s, torch.float32), torch.float32)
