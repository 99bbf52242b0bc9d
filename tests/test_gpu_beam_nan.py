"""Beams whose score so far is NaN: they count as beams without a score."""
import numpy as np
import pytest
import torch

from tests.test_gpu_beam import call, draw, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,Kout", [(1, 4), (2, 32), (5, 8)])
@pytest.mark.parametrize("ended", [False, True])
def test_candidates_of_a_nan_score_are_the_lowest_tokens(cuda_dev, K, Kout, ended):
    logits, cum = draw(2, K, 3000, "bf16", 80 + K)
    cum[:, 0] = float("-inf")
    cum[1] = float("-inf")
    bad = torch.where(torch.isinf(cum), torch.full_like(cum, float("nan")), cum)
    finished = torch.zeros(2, K, dtype=torch.int32)
    finished[:, 0] = int(ended)
    got, want = call(logits.cuda(), bad, finished, 50, Kout), reference(logits, cum, finished, 50, Kout)
    for g, w in zip(got[1:], want[1:]):
        assert np.array_equal(g.numpy(), w)
    assert np.array_equal(np.isneginf(got[0].numpy()), np.isneginf(want[0])) and not torch.isnan(got[0]).any()
