"""Cosines and sines of the rotation by their own size: slow pairs at near positions, where a sine is a small number, and
far positions next to whole and quarter turns."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_rope import near

pytestmark = pytest.mark.gpu

#          base, scaling, factor, rotated dims
SLOW = [(1e4, 0, 1.0, 128), (5e5, 1, 8.0, 128), (5e6, 1, 4.0, 128), (5e5, 2, 16.0, 64), (1e6, 3, 32.0, 256), (1e7, 4, 8.0, 96)]


def turns(pos, steps):
    """(quarter turns, radians left in [-pi / 4, pi / 4]) of positions times steps modulo a turn, from whole numbers."""
    q, rest = [], []
    for p in pos:
        for s in steps:
            part = p * (s % (1 << 64)) % (1 << 64)
            k = (part + (1 << 61)) >> 62
            q.append(k % 4)
            rest.append((part - (k << 62)) / 2.0 ** 64 * 2 * math.pi)  # (rounded once: 2^-53 of itself, the products 2^-52)
    return np.array(q).reshape(len(pos), -1), np.array(rest).reshape(len(pos), -1)


@pytest.mark.parametrize("case", SLOW, ids=str)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("one", [0, 1])
def test_of_one_element(cuda_dev, case, layout, one):
    """A pair (x, 0) or (0, x): an output is one product, off by less than a step (2^-23) of the cosine or sine and half
    a step of the product (2^-24), relative to itself, before it is rounded to fp16."""
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    base, scaling, factor, rot = case
    steps, _ = LT.lucetree_rope_steps(rot, base, scaling=scaling, factor=factor, orig_ctx=4096, low=1, high=32)
    g = np.random.default_rng(rot)
    pos = [1, -1, 2, 3, 5, 63, 100, 1000, 4097, 131071, -131071, 2 ** 31 - 1, -2 ** 31] + g.integers(0, 2 ** 20, 200).tolist()
    N, h = len(pos), rot // 2
    q = torch.zeros(1, N, 1, rot, dtype=torch.float16)
    at = (slice(one * h, (one + 1) * h) if layout == 0 else slice(one, None, 2), slice(h, None) if layout == 0 else slice(1, None, 2),
          slice(0, h) if layout == 0 else slice(0, None, 2))
    x = 60000.0
    q[..., at[0]] = x
    x = float(q[..., at[0]].max())
    out = [torch.empty(1, N, 1, rot, dtype=torch.float16, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    LT.lucetree_rope(q.cuda(), q.cuda(), steps.cuda(), layout, *out, status,
                     positions=torch.tensor([pos], dtype=torch.int32, device="cuda"))
    quarter, rest = turns(pos, steps.tolist())
    c, s = np.cos(rest), np.sin(rest)
    cos, sin = np.choose(quarter, [c, -s, -c, s]), np.choose(quarter, [s, c, -s, -c])
    want = torch.zeros(N, rot, dtype=torch.float64)
    want[:, at[2]] = torch.from_numpy(x * (-sin if one else cos))
    want[:, at[1]] = torch.from_numpy(x * (cos if one else sin))
    for o in out:
        near(o[0, :, 0], want, (2.0 ** -22 - 2.0 ** -24) * want.abs())
