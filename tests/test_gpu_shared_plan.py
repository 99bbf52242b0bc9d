"""The plan of a batch that shares prefixes: the common pages against the page tables, and its pieces, each tile of
each segment in exactly one of them."""
import numpy as np
import pytest
import torch

from tests.shared_cases import PAGE, batch, check_plan, common

pytestmark = pytest.mark.gpu


def make_plan(ctx, start, table, pages, N, Hq, Hkv, D, stream=None):
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    B, groups = len(ctx), len(start) - 1
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    plan = torch.full((LT.lucetree_shared_plan_bytes(B, N, Hq, Hkv, D, groups),), 0x77, dtype=torch.uint8, device="cuda")
    shared = torch.full((groups,), -5, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    LT.lucetree_shared_plan(i32(table), i32(ctx), i32(start), N, Hq, Hkv, D, pages, shared, plan, status, stream=stream)
    torch.cuda.synchronize()
    return plan, shared, int(status.item())


def check(groups, N, Hq, Hkv, D, seed=0, **kw):
    ctx, start, table, pages = batch(groups, N, seed, **kw)
    plan, shared, status = make_plan(ctx, start, table, pages, N, Hq, Hkv, D)
    assert status == 0
    assert shared.tolist() == common(ctx, start, table, pages)
    return check_plan(plan, ctx, start, table, pages, N, Hq, Hkv, D)


BATCHES = [
    ([(0, [0])], 1, 1, 1),
    ([(8, [512, 600, 530, 575])], 1, 8, 2),
    ([(8, [512, 600, 530, 575])], 22, 24, 4),
    ([(200, [13000 + 17 * i for i in range(32)])], 1, 24, 4),
    ([(64, [4200, 4300, 5000]), (0, [9000]), (3, [200, 210]), (0, []), (17, [1100] * 9)], 5, 15, 5),
    ([(0, [L]) for L in (0, 1, 63, 64, 65, 20000, 300)], 3, 6, 3),
    ([(40, [2600] * 8) for _ in range(24)], 1, 24, 4),
    ([(1, [64, 64])], 1, 4, 4),
    ([(100, [6400] * 40)], 64, 12, 2),
    ([(100, [6401, 100000])], 1, 2, 1),
    ([(31, [1984 + i for i in range(7)]), (33, [2112] * 3)], 7, 128, 1),
]


@pytest.mark.parametrize("i", range(len(BATCHES)))
@pytest.mark.parametrize("D", [128, 256])
def test_pieces(cuda_dev, i, D):
    check(*BATCHES[i], D, seed=i)


def test_many_batches(cuda_dev):
    rng = np.random.default_rng(3)
    for seed in range(60):
        groups = []
        for _ in range(rng.integers(1, 12)):
            both = int(rng.integers(0, 60))
            groups.append((both, [int(both * PAGE + rng.integers(0, 700)) for _ in range(rng.integers(1, 14))]))
        Hkv = int(rng.integers(1, 6))
        check(groups, int(rng.integers(1, 65)), Hkv * int(rng.integers(1, 9)), Hkv, 128, seed=seed)


def test_hundreds_of_sequences(cuda_dev):
    rng = np.random.default_rng(5)
    check([(int(x), [int(x) * PAGE + int(y) for y in rng.integers(0, 300, 7)]) for x in rng.integers(0, 20, 150)],
          2, 4, 2, 128, seed=1)


def test_rows_that_differ_early_and_entries_that_name_no_page(cuda_dev):
    ctx, start, table, pages = batch([(20, [1300, 1400, 1350])], 1)
    for col, row, value in ((13, 2, 0), (13, 0, -1), (7, 1, 10 ** 6)):
        t = table.copy()
        t[row, col] = value if value != 0 else t[row, col + 1]
        plan, shared, status = make_plan(ctx, start, t, pages, 1, 8, 2, 128)
        assert status == 0 and shared.tolist() == [col] == common(ctx, start, t, pages)
    t = table.copy()
    t[:, 9] = pages  # the same in all rows, but no page
    assert make_plan(ctx, start, t, pages, 1, 8, 2, 128)[1].tolist() == [9]


def test_a_sequence_that_is_shorter_than_the_prefix(cuda_dev):
    ctx, start, table, pages = batch([(20, [1300, 1400, 1350])], 1)
    ctx[1] = 640 + 63
    plan, shared, status = make_plan(ctx, start, table, pages, 1, 8, 2, 128)
    assert status == 0 and shared.tolist() == [10]
    check_plan(plan, ctx, start, table, pages, 1, 8, 2, 128)


@pytest.mark.parametrize("start", [(0, 2, 1, 4), (1, 2, 3, 4), (0, 1, 2, 3), (0, 1, 2, 9), (0, -1, 2, 4)])
def test_bad_groups_share_nothing(cuda_dev, start):
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    ctx, _, table, pages = batch([(20, [1300, 1400, 1350, 1290])], 1)
    plan, shared, status = make_plan(ctx, np.array(start), table, pages, 1, 8, 2, 128)
    assert status == LT.DEV_BAD_ROW and shared.tolist() == [0, 0, 0]


def test_bad_lengths_are_empty(cuda_dev):
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    ctx, start, table, pages = batch([(20, [1300, 1400, 1350, 1290])], 1)
    for L in (-1, table.shape[1] * PAGE + 1):
        bad = ctx.copy()
        bad[2] = L
        plan, shared, status = make_plan(bad, start, table, pages, 1, 8, 2, 128)
        assert status == LT.DEV_BAD_CTX and shared.tolist() == [0]
        bad[2] = 0
        check_plan(plan, bad, start, table, pages, 1, 8, 2, 128)
