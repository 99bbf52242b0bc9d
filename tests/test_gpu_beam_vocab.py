"""Beam selection over the largest vocabularies that it takes."""
import pytest
import torch

from tests.test_gpu_beam import _lt, call


def test_as_many_chunks_as_for_half_the_vocabulary():
    LT = _lt()
    for batch, K in ((1, 1), (2, 2)):
        assert LT.lucetree_beam_select_workspace(batch, K, 1, 2 ** 31 - 1) == \
            LT.lucetree_beam_select_workspace(batch, K, 1, 2 ** 30)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,short", [("bfloat16", 0), ("bfloat16", 6), ("float32", 0), ("float32", 27)])
def test_elements_next_to_two_to_the_31(cuda_dev, dtype, short):
    V = 2 ** 31 - 1 - short
    logits = torch.zeros(1, 1, V, dtype=getattr(torch, dtype), device="cuda")
    best = [V - 1, 5, V // 8 * 8 - 1, V - 3, 0]
    for i, v in enumerate(best):
        logits[0, 0, v] = 30 - i
    score, token, row, fin = call(logits, torch.zeros(1, 1), None, V - 1, 6)
    assert token.tolist() == [best + [1]] and row.tolist() == [[0] * 6] and fin.tolist() == [[1, 0, 0, 0, 0, 0]]
    # sum = e^30 (1 + 1/e + ..) + 2^31: relative to fp32's terms of 2^31 in e^30 = 1e13
    want = torch.tensor([30.0 - i for i in range(5)] + [0.0], dtype=torch.float64)
    want -= torch.log(torch.exp(want[:5]).sum() + (V - 5))
    # a thread adds up at most V / (4 x SMs x 256) = 14,000 ones after a term of e^30 and loses at most half a step of the
    # sum with each: 14,000 x 2^-24 of the logarithm's argument, and 16 x 2^-24 as for other vocabularies
    assert ((score[0].double() - want).abs() <= 14016 * 2.0 ** -24 + 2.0 ** -24 * want.abs()).all()
