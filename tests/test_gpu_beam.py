"""Beam selection against its definition in 64 bits: exact whole numbers, ties
to the lower beam and token, finished and dead beams, masked vocabularies, odd
sizes, alignments and strides."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _lt():
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    return LT


def reference(logits, cum, finished, eos, Kout):
    x, cum = logits.double().numpy(), cum.double().numpy()
    B, K, V = x.shape
    out = [np.zeros((B, Kout)), *(np.zeros((B, Kout), np.int64) for _ in range(3))]
    for b in range(B):
        score = np.full((K, V), -np.inf)
        for k in range(K):
            if finished is not None and finished[b, k]:
                if 0 <= eos < V:
                    score[k, eos] = cum[b, k]
            elif np.isfinite(x[b, k]).any() and np.isfinite(cum[b, k]):
                m = x[b, k].max()
                score[k] = x[b, k] - (m + np.log(np.exp(x[b, k] - m).sum())) + cum[b, k]
        order = np.argsort(-score.reshape(-1), kind="stable")[:Kout]
        out[0][b] = score.reshape(-1)[order]
        out[1][b], out[2][b] = order % V, b * K + order // V
        for j, i in enumerate(order):
            ended = finished is not None and bool(finished[b, i // V])
            out[3][b, j] = int(ended or i % V == eos)
    return out


def call(logits, cum, finished, eos, Kout, done=True, ws=None):
    LT = _lt()
    B, K, V = logits.shape
    i32 = lambda: torch.full((B, Kout), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    score, token, row, fin = torch.full((B, Kout), float("nan"), device="cuda"), i32(), i32(), i32()
    if ws is None:
        ws = torch.empty(LT.lucetree_beam_select_workspace(B, K, Kout, V), dtype=torch.uint8, device="cuda")
        ws.fill_(0xFF)
    LT.lucetree_beam_select(logits, cum.cuda(), None if finished is None else finished.cuda(), eos, score, token, row,
                            fin if done else None, ws)
    torch.cuda.synchronize()
    return score.cpu(), token.cpu(), row.cpu(), fin.cpu()


def check(logits, cum, finished, eos, Kout, dev=None):
    """dev: the device logits, where their layout differs from the host's."""
    got = call(logits.cuda() if dev is None else dev, cum, finished, eos, Kout)
    want = reference(logits, cum, finished, eos, Kout)
    for g, w in zip(got[1:], want[1:]):
        assert np.array_equal(g.numpy(), w)
    g, w = got[0].double().numpy(), want[0]
    assert np.array_equal(np.isneginf(g), np.isneginf(w))
    g, w = g[~np.isneginf(w)], w[~np.isneginf(w)]
    # the sum's fp32 terms are off by a few 2^-24 each (difference, product, exponential of 2 ulp) and so is its
    # logarithm; one more rounding of the score
    assert np.all(np.abs(g - w) <= 16 * 2.0 ** -24 + 2.0 ** -24 * np.abs(w))


def draw(B, K, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(B, K, V, generator=g)).to(TYPES[dtype]), -10 * torch.rand(B, K, generator=g)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,K,Kout,V", [(1, 1, 1, 1), (1, 1, 3, 3), (2, 3, 5, 7), (1, 4, 4, 100), (3, 2, 32, 33),
                                        (1, 32, 32, 1000), (2, 5, 7, 4097), (5, 8, 8, 30011), (1, 1, 8, 151936),
                                        (2, 31, 17, 20001)])
def test_matches_the_definition(cuda_dev, dtype, B, K, Kout, V):
    logits, cum = draw(B, K, V, dtype, seed=B + K + V)
    check(logits, cum, None, -1, Kout)


@pytest.mark.parametrize("dtype", TYPES)
def test_finished_dead_and_masked(cuda_dev, dtype):
    logits, cum = draw(6, 5, 2051, dtype, seed=3)
    g = torch.Generator().manual_seed(4)
    logits.masked_fill_(torch.rand(6, 5, 2051, generator=g) < 0.97, float("-inf"))
    logits[1, 2] = float("-inf")                       # no token left
    logits[5] = float("-inf")
    finished = (torch.rand(6, 5, generator=g) < 0.4).int()
    finished[2] = torch.tensor([0, -3, 1 << 30, 0, 1], dtype=torch.int32)  # any non-zero value
    cum[0, 1:] = float("-inf")                         # the first step of a search
    cum[3] = float("-inf")
    finished[4] = 1
    for eos in (0, 17, 2050, -1, 2051):
        check(logits, cum, finished, eos, 8)
        check(logits, cum, finished, eos, 32)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_lower_beam_and_token(cuda_dev, dtype):
    for V in (64, 5003):
        logits = torch.zeros(2, 4, V, dtype=TYPES[dtype])
        logits[0, :, 5::7] = 2.0                       # many equal best tokens, equal rows
        logits[0, 2, 6] = -0.0
        logits[1] = torch.randint(0, 3, (4, V), generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
        logits[1, 1:] = logits[1, 0]                   # the same sums in every row
        check(logits, torch.full((2, 4), -1.5), None, 3, 32)


def test_large_and_far_logits(cuda_dev):
    logits, cum = draw(2, 3, 9001, "f32", seed=8, spread=1e3)
    check(logits + 5e4, cum, None, -1, 8)
    logits = torch.linspace(-3e38, 3e38, 4099, dtype=torch.float64).float().expand(1, 2, 4099).contiguous()
    check(logits, torch.tensor([[-1.0, -2.0]]), None, -1, 2)


def test_sorted_rows_change_the_list_most(cuda_dev):
    up = torch.arange(20000, dtype=torch.float32)[None, None] * 1e-3
    check(up.contiguous(), torch.zeros(1, 1), None, -1, 32)
    check(up.flip(-1).contiguous(), torch.zeros(1, 1), None, -1, 32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset,stride", [(0, 1003), (1, 1003), (3, 1024), (5, 1001), (7, 1011)])
def test_rows_of_any_alignment_and_stride(cuda_dev, dtype, offset, stride):
    B, K, V = 2, 3, 1001
    logits, cum = draw(B, K, V, dtype, seed=offset)
    flat = torch.full((offset + B * K * stride,), 1e4, device="cuda").to(TYPES[dtype])  # larger than any logit
    dev = flat[offset:].view(B * K, stride)[:, :V].unflatten(0, (B, K))
    dev.copy_(logits)
    check(logits, cum, None, -1, 6, dev=dev)


def test_short_rows_of_any_alignment(cuda_dev):
    for V in range(1, 24):
        flat = torch.full((8 + 4 * 25,), 1e4, dtype=torch.float16, device="cuda")
        logits, cum = draw(1, 3, V, "f16", seed=V)
        for offset in range(8):
            dev = flat[offset:offset + 75].view(3, 25)[:, :V][None]
            dev.copy_(logits)
            check(logits, cum, None, 1, min(9, 3 * V), dev=dev)


def test_equal_rows_tie_wherever_they_lie(cuda_dev):
    # rows 1003 elements apart start on every 4-byte boundary: their sums have to be the same bits
    for dtype in TYPES:
        flat = torch.zeros(2 * 7 * 1003 + 8, device="cuda").to(TYPES[dtype])
        row, _ = draw(1, 1, 1000, dtype, seed=4)
        for offset in range(4):
            dev = flat[offset:offset + 2 * 7 * 1003].view(14, 1003)[:, :1000].unflatten(0, (2, 7))
            dev.copy_(row.expand(2, 7, 1000))
            check(row.expand(2, 7, 1000).contiguous(), torch.full((2, 7), -2.0), None, -1, 30, dev=dev)


def test_nan_logits_stay_inside_the_outputs(cuda_dev):
    # outside the contract, but what comes back still names rows and tokens that exist
    for bits in (0x7FC00000, 0xFFC00000 - (1 << 32)):
        nan = torch.tensor([bits], dtype=torch.int32).view(torch.float32)
        logits = nan.expand(2 * 3 * 70).reshape(2, 3, 70).contiguous()
        logits[1, 1, 5] = 1.0
        score, token, row, fin = call(logits.cuda(), torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int32), 5, 32)
        assert ((token >= 0) & (token < 70)).all() and (row // 3 == torch.arange(2)[:, None]).all()


def test_scores_and_flags_updated_in_place(cuda_dev):
    LT = _lt()
    B, K, V = 5, 6, 3001
    logits, cum = draw(B, K, V, "bf16", seed=11)
    finished = (torch.rand(B, K, generator=torch.Generator().manual_seed(2)) < 0.3).int()
    want = reference(logits, cum, finished, 9, K)
    c, f, x = cum.cuda(), finished.cuda(), logits.cuda()
    token, row = (torch.empty(B, K, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(LT.lucetree_beam_select_workspace(B, K, K, V), dtype=torch.uint8, device="cuda")
    LT.lucetree_beam_select(x, c, f, 9, c, token, row, f, ws)
    assert np.array_equal(token.cpu().numpy(), want[1]) and np.array_equal(row.cpu().numpy(), want[2])
    assert np.array_equal(f.cpu().numpy(), want[3])
    assert np.all(np.abs(c.double().cpu().numpy() - want[0]) <= 16 * 2.0 ** -24 + 2.0 ** -24 * np.abs(want[0]))


def test_without_the_optional_outputs(cuda_dev):
    logits, cum = draw(2, 2, 500, "f32", seed=1)
    got = call(logits.cuda(), cum, None, 4, 3, done=False)
    want = reference(logits, cum, None, 4, 3)
    assert np.array_equal(got[1].numpy(), want[1]) and (got[3] == -7).all()


def test_captured_replayed_and_two_streams_at_once(cuda_dev):
    LT = _lt()
    B, K, V = 2, 4, 33333
    sets = [draw(B, K, V, "bf16", seed=s) for s in (1, 2)]
    want = [reference(x, c, None, 5, 4) for x, c in sets]
    dev = [(x.cuda(), c.cuda()) for x, c in sets]
    outs = [[torch.empty(B, 4, dtype=t, device="cuda") for t in (torch.float32,) + (torch.int32,) * 3] for _ in sets]
    ws = [torch.empty(LT.lucetree_beam_select_workspace(B, K, 4, V), dtype=torch.uint8, device="cuda") for _ in sets]
    go = lambda i: LT.lucetree_beam_select(*dev[i], None, 5, *outs[i], ws[i])  # noqa: E731
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                go(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(outs[i][1].cpu().numpy(), want[i][1])
        assert np.array_equal(outs[i][2].cpu().numpy(), want[i][2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(0)
    for i in (1, 0):
        dev[0][0].copy_(sets[i][0])
        dev[0][1].copy_(sets[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(outs[0][1].cpu().numpy(), want[i][1])


@pytest.mark.parametrize("step,K,Kout", [(8, 32, 32), (8, 16, 32), (4, 32, 17), (1, 32, 32)])
def test_good_candidates_crowded_into_some_chunks(cuda_dev, step, K, Kout):
    """Every `step`-th chunk of a request holds all its good candidates, more than Kout each."""
    V, sms = 50000, torch.cuda.get_device_properties(0).multi_processor_count
    chunks = max(1, 4 * sms // K)  # (other cuts are no less right, only easier)
    logits, cum = draw(1, K, V, "f32", 41)
    g = torch.Generator().manual_seed(42)
    for i in range(0, K * chunks, step):
        k, first = divmod(i, chunks)
        first = V // 4 * first // chunks * 4 + 8
        logits[0, k, first:first + 120:3] = 40 + 5 * torch.rand(40, generator=g)
    check(logits, cum, None, -1, Kout)


@pytest.mark.parametrize("Kout", [1, 2, 3, 4, 9, 16])
def test_one_beam_far_ahead(cuda_dev, Kout):
    """All candidates come from one row."""
    logits, cum = draw(3, 6, 20000, "bf16", 43)
    cum[:, 4] += 1000
    check(logits, cum, None, -1, Kout)


def test_equal_scores_everywhere(cuda_dev):
    """One value in every row: the order is that of beams and tokens alone."""
    check(torch.full((2, 8, 9000), 0.5), torch.full((2, 8), -1.0), None, -1, 32)


@pytest.mark.parametrize("B,K,V,live", [(1, 4, 4096, 1), (3, 5, 3000, 2), (4, 8, 20001, 0), (4, 8, 20001, 32), (40, 8, 5000, 37),
                                        (76, 8, 1100, 300), (100, 8, 700, 500), (1, 32, 60000, 3)])
def test_any_number_of_ended_and_dead_beams(cuda_dev, B, K, V, live):
    """Live rows anywhere among ended and dead ones, up to more rows than run at once."""
    logits, cum = draw(B, K, V, "bf16", 50 + live)
    g = torch.Generator().manual_seed(51 + live)
    order = torch.randperm(B * K, generator=g)[: B * K - live]
    finished = torch.zeros(B * K, dtype=torch.int32)
    finished[order[::2]] = 1
    cum.view(-1)[order[1::2]] = float("-inf")
    check(logits, cum, finished.view(B, K), 7, min(K, 8))


def test_scores_that_are_not_numbers_come_last(cuda_dev):
    """A beam whose score so far is NaN counts as -inf; the others are chosen as without it."""
    logits, cum = draw(2, 5, 3000, "f16", 60)
    bad = cum.clone()
    bad[:, 3] = float("nan")
    cum[:, 3] = float("-inf")
    got, want = call(logits.cuda(), bad, None, -1, 6), reference(logits, cum, None, -1, 6)
    assert np.array_equal(got[1].numpy(), want[1]) and np.array_equal(got[2].numpy(), want[2])
    assert not torch.isnan(got[0]).any()
