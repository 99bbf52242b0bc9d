"""Batches whose groups are of unlike size: how often a group's common pages are gone through, by the group's own rows, and
the attention of such batches against the formula."""
import numpy as np
import pytest
import torch

from tests import shared_cases
from tests.shared_cases import PAGE, batch, check_plan, common
from tests.test_gpu_attention_shared import P_STEP, make, near, reference
from tests.test_gpu_shared_edges import Call
from tests.test_gpu_shared_plan import make_plan

pytestmark = pytest.mark.gpu

read_plan = shared_cases.read_plan


def cap_of(B, groups, N, G):
    """Nodes of a block at most: rows of one CTA, or of two where the mean group has more than one's."""
    return 128 // G * (2 if -(-B // groups) * N * G > 128 else 1)


def uneven(monkeypatch, ctx, start, table, pages, N, Hq, Hkv, D):
    """The plan, checked piece by piece, with blocks of any size up to the most: a group's rows go through fewer than 60
    common pages more than they would in the fewest blocks.  -> (blocks of each group, its pages that are read once)."""
    B, groups, G = len(ctx), len(start) - 1, Hq // Hkv
    cap = cap_of(B, groups, N, G)
    monkeypatch.setattr(shared_cases, "read_plan", lambda *a: {**read_plan(*a), "NPG": cap})
    plan, shared, status = make_plan(ctx, start, table, pages, N, Hq, Hkv, D)
    both = common(ctx, start, table, pages)
    assert status == 0 and shared.tolist() == both
    p = check_plan(plan, ctx, start, table, pages, N, Hq, Hkv, D)
    blocks = [int((p["blk"][:int(p["head"][0, 10]), 0] == g).sum()) for g in range(groups)]
    used = p["grp"][:groups, 0].tolist()
    least = [-(-int(z - a) * N // cap) for a, z in zip(start[:-1], start[1:])]
    for g in range(groups):
        n = int(start[g + 1] - start[g])
        if both[g] and n > 1:
            assert ((blocks[g] if used[g] else n * p["NG"]) - least[g]) * both[g] < 60
    return blocks, used


def fork(pages, n, alone, own=100):
    """One group of n sequences under `pages` common pages, beside single ones."""
    return [(pages, [pages * PAGE + own + 7 * i for i in range(n)])] + [(0, [300 + i]) for i in range(alone)]


#       common, sequences, beside, N, Hq, Hkv: blocks of the large group.  (40: 2,048 nodes by 41, the mean group's share,
#       are 50 blocks where 49 would do, and stay; 3: a block holds one sequence, so nothing is read once.)
FORKS = {(256, 32, 32, 1, 24, 4): 2, (256, 32, 32, 22, 24, 4): 17, (40, 32, 5, 64, 24, 4): 50, (64, 200, 200, 1, 24, 4): 10,
         (20, 300, 40, 1, 4, 4): 3, (20, 300, 40, 5, 4, 4): 12, (3, 60, 61, 2, 128, 1): 60, (30, 17, 100, 13, 15, 5): 6}


@pytest.mark.parametrize("case", list(FORKS), ids=str)
@pytest.mark.parametrize("D", [128, 256])
def test_a_large_group_beside_single_sequences(cuda_dev, monkeypatch, case, D):
    pages, n, alone, N, Hq, Hkv = case
    ctx, start, table, total = batch(fork(pages, n, alone), N)
    blocks, used = uneven(monkeypatch, ctx, start, table, total, N, Hq, Hkv, D)
    assert blocks[0] == FORKS[case] and used[0] == (0 if pages == 3 else pages)


def test_groups_of_any_sizes(cuda_dev, monkeypatch):
    rng = np.random.default_rng(8)
    for seed in range(60):
        groups = []
        for _ in range(rng.integers(1, 20)):
            both, n = int(rng.integers(0, 40)), int(2 ** rng.uniform(0, 7))
            groups.append((both, [int(both * PAGE + rng.integers(0, 400)) for _ in range(n)]))
        Hkv, N = int(rng.integers(1, 5)), int(2 ** rng.uniform(0, 6.02))
        ctx, start, table, total = batch(groups, N, seed)
        uneven(monkeypatch, ctx, start, table, total, N, Hkv * int(rng.integers(1, 9)), Hkv, 128)


#     groups,                                                                      N,  Hq, Hkv, D, dtype
ATTEND = [
    (fork(10, 32, 32), 1, 24, 4, 256, "bf16"), (fork(8, 20, 20), 22, 24, 4, 256, "bf16"), (fork(8, 20, 20), 22, 12, 2, 128, "f16"),
    (fork(6, 40, 50), 1, 128, 1, 128, "bf16"), (fork(5, 300, 40), 1, 4, 4, 128, "f16"),
    (fork(4, 9, 3) + fork(7, 30, 40), 5, 6, 2, 256, "f16"), (fork(3, 24, 30), 64, 8, 2, 128, "bf16"),
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
@pytest.mark.parametrize("out", ["f32", "same"])
def test_attention_of_uneven_groups(cuda_dev, i, out):
    s = make(*ATTEND[i], seed=50 + i)
    t = torch.float32 if out == "f32" else s["q"].dtype
    got, lse, status = Call(s, t).run()
    assert status == 0
    near(got, lse, reference(s, p_step=P_STEP[t]))


def test_a_captured_step_whose_groups_change(cuda_dev):
    """Plan and attention captured with even groups, replayed with one large group: which cut is taken is decided on the
    device."""
    even = make([(10, [700, 650, 800, 641]) for _ in range(10)], 1, 24, 4, 128, "bf16", seed=3)
    large = make(fork(30, 31, 9), 1, 24, 4, 128, "bf16", seed=4)
    B, G = 40, 10
    assert large["q"].shape == even["q"].shape and large["group_start"].numel() == even["group_start"].numel() == G + 1
    wide = max(s["page_table"].shape[1] for s in (even, large))
    pages = max(s["k_pool"].shape[0] for s in (even, large))
    for s in (even, large):
        table = torch.full((B, wide), -1, dtype=torch.int32)
        table[:, :s["page_table"].shape[1]] = s["page_table"]
        s["page_table"] = table
        for k in ("k_pool", "v_pool"):
            s[k] = torch.cat([s[k], torch.full((pages - s[k].shape[0], *s[k].shape[1:]), float("nan"), dtype=s[k].dtype)])
    c = Call(even)
    c.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.make_plan()
        c.attend()
    for s in (large, even, large):
        for k, v in s.items():
            c.d[k].copy_(v)
        c.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0 and c.shared.tolist() == ([30] + [0] * 9 if s is large else [10] * 10)
        near(c.out.cpu(), c.lse.cpu(), reference(s, p_step=P_STEP[torch.float32]))
        assert int(c.plan.cpu().numpy().view(np.int32)[10]) == (11 if s is large else 10)  # blocks
