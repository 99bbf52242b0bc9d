"""Beams that have ended or live on with a score of -infinity or NaN."""
import numpy as np
import pytest
import torch

from tests.test_gpu_beam import call, check, draw, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,Kout", [(1, 4), (1, 32), (3, 4), (8, 8)])
@pytest.mark.parametrize("eos", [0, 2, 50, 2999, -1])
def test_an_ended_beam_without_a_score_ties_like_any_other(cuda_dev, K, Kout, eos):
    logits, cum = draw(2, K, 3000, "bf16", 70 + K)
    cum[:] = float("-inf")
    finished = torch.zeros(2, K, dtype=torch.int32)
    finished[:, 0] = 1
    check(logits, cum, finished, eos, Kout)
    finished[1] = 1
    check(logits, cum, finished, eos, Kout)
