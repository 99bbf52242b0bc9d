"""Tree-verify attention of batches that share prefixes against the formula in 64 bits: groups of one, few and many
sequences, prefixes from none to long, row blocks that end inside a sequence, lengths of zero and one, anything at all
behind a sequence's end."""
import numpy as np
import pytest
import torch

from tests.shared_cases import PAGE, TYPES, batch

pytestmark = pytest.mark.gpu

P_STEP = {torch.float32: 2.0 ** -11, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def _lt():
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    return LT


def make(groups, N, Hq, Hkv, D, dtype, tree="random", seed=0, junk=float("nan")):
    """Inputs with `junk` behind every sequence's last key."""
    rng, g, t = np.random.default_rng(seed), torch.Generator().manual_seed(seed), TYPES[dtype]
    ctx, start, table, pages = batch(groups, N, seed)
    B = len(ctx)
    r = lambda *s: torch.randn(*s, generator=g).to(t)  # noqa: E731
    pools = [r(pages, Hkv, PAGE, D) for _ in range(2)]
    filled = np.zeros(pages * PAGE, bool)
    for b, L in enumerate(ctx):
        pos = np.arange(L)
        filled[table[b, pos // PAGE] * PAGE + pos % PAGE] = True
    page, slot = np.nonzero(~filled.reshape(pages, PAGE))
    for pool in pools:
        pool[torch.from_numpy(page), :, torch.from_numpy(slot)] = junk
    parent = np.full((B, N), -1, np.int64)
    for i in range(1, N):
        parent[:, i] = i - 1 if tree == "chain" else rng.integers(-1, i, size=B)
    sees = np.zeros((B, N, N), bool)
    for i in range(N):
        sees[:, i, i] = True
        for b in range(B):
            if parent[b, i] >= 0:
                sees[b, i] |= sees[b, parent[b, i]]
    anc = (sees.astype(np.uint64) << np.arange(N, dtype=np.uint64)).sum(-1, dtype=np.uint64)
    return dict(q=r(B, N, Hq, D), k_pool=pools[0], v_pool=pools[1], page_table=torch.from_numpy(table),
                ctx_len=torch.from_numpy(ctx), group_start=torch.from_numpy(start), k_tree=r(B, N, Hkv, D),
                v_tree=r(B, N, Hkv, D), anc_mask=torch.from_numpy(anc.view(np.int64)), sees=torch.from_numpy(sees))


def reference(s, scale=None, p_step=2.0 ** -11):
    """(out, lse, bound, lse_bound): the formula in 64 bits, and how far a correct kernel's output may be from it.

    P is rounded to fp16 (half a step: 2^-11 of each term; with a bf16 output to bf16: 2^-8) relative to a shift that
    lies within the factor 2^8 of the row's largest term, so a term below 2^-24 of it is off by at most 2^-25.  A score
    is a sum of D exact products in fp32: off by at most D 2^-24 sum|q k| scale, which moves each term by that
    fraction; 2^-20 more covers the exponential, the sums and the shifts."""
    d = {k: v.cuda() for k, v in s.items()}
    q, (B, N, Hq, D) = d["q"].double(), s["q"].shape
    Hkv = s["k_tree"].shape[2]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        L = int(s["ctx_len"][b])
        at = torch.arange(L, device="cuda")
        page = d["page_table"][b][at // PAGE].long()
        on = torch.cat([torch.ones(N, L, dtype=torch.bool, device="cuda"), d["sees"][b]], 1)[:, None]
        for g in range(Hkv):
            k = torch.cat([d["k_pool"][page, g, at % PAGE], d["k_tree"][b, :, g]]).double()
            v = torch.cat([d["v_pool"][page, g, at % PAGE], d["v_tree"][b, :, g]]).double()
            hs = slice(g * G, (g + 1) * G)
            x = torch.where(on, q[b, :, hs] @ k.T * scale, float("-inf"))
            lse[b, :, hs] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[b, :, hs, None])
            out[b, :, hs] = p @ v
            err = (D * 2.0 ** -24 * abs(scale) * torch.where(on, q[b, :, hs].abs() @ k.abs().T, 0.0)).amax(-1, keepdim=True) + 2.0 ** -20
            bound[b, :, hs] = (p_step + 2 * err) * (p @ v.abs()) + 2.0 ** -25 * p.amax(-1, keepdim=True) * v.abs().sum(0)
            lse_bound[b, :, hs] = err[..., 0] + 2.0 ** -24 * lse[b, :, hs].abs()
    return out.cpu(), lse.cpu(), bound.cpu(), lse_bound.cpu()


def call(s, out_dtype, lse=True, scale=None, stream=None, table=None, anc=None, plan_table=None):
    LT = _lt()
    d = {k: v.cuda() for k, v in s.items()}
    (B, N, Hq, D), Hkv, groups = s["q"].shape, s["k_tree"].shape[2], s["group_start"].numel() - 1
    out = torch.full((B, N, Hq, D), float("nan"), dtype=out_dtype, device="cuda")
    lse_t = torch.full((B, N, Hq), float("nan"), device="cuda") if lse else None
    status, shared = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(groups, dtype=torch.int32, device="cuda")
    plan = torch.empty(LT.lucetree_shared_plan_bytes(B, N, Hq, Hkv, D, groups), dtype=torch.uint8, device="cuda")
    ws = torch.empty(LT.lucetree_verify_attn_shared_workspace(B, N, Hq, Hkv, D, groups), dtype=torch.uint8, device="cuda")
    ws.fill_(0x7F)  # garbage (3.4e38 as fp32): a partial read before it is written shows
    table = d["page_table"] if table is None else table
    LT.lucetree_shared_plan(table if plan_table is None else plan_table, d["ctx_len"], d["group_start"], N, Hq, Hkv, D,
                            d["k_pool"].shape[0], shared, plan, status, stream=stream)
    LT.lucetree_verify_attn_shared(d["q"], d["k_pool"], d["v_pool"], table, d["ctx_len"], d["k_tree"], d["v_tree"],
                                   d["anc_mask"] if anc is None else anc, groups, plan, out, status, ws, lse=lse_t,
                                   scale=scale, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), None if lse_t is None else lse_t.cpu(), int(status.item())


def near(out, lse, ref, rows=slice(None)):
    want, want_lse, bound, lse_bound = (t[rows] for t in ref)
    out = out[rows]
    bound = bound + (0 if out.dtype == torch.float32 else torch.finfo(out.dtype).eps / 2) * (want.abs() + bound)
    assert bool(torch.isfinite(out).all())
    far = float(((out.double() - want).abs() / (bound + 2.0 ** -24 * want.abs())).max())
    assert far <= 1
    if lse is not None:
        assert bool(((lse[rows].double() - want_lse).abs() <= lse_bound).all())


def check(s, out_dtype, **kw):
    out, lse, status = call(s, out_dtype, **kw)
    assert status == 0
    near(out, lse, reference(s, kw.get("scale"), P_STEP[out_dtype]))


#     (pages in common, lengths) ...,                                        N,  Hq, Hkv, D,  dtype
CASES = [
    ([(8, [512, 600, 530, 575])],                                             1,  8,  2, 128, "f16"),
    ([(8, [512, 600, 530, 575])],                                             8,  8,  2, 128, "f16"),
    ([(0, [0])],                                                              1,  1,  1, 128, "bf16"),
    ([(0, [0, 1, 63, 64, 65, 127, 300])],                                     3,  4,  2, 128, "bf16"),
    ([(0, [L]) for L in (0, 1, 63, 64, 65, 2000, 300)],                       5,  6,  3, 256, "f16"),
    ([(20, [1280, 1281, 1343, 1344, 1345, 1300, 1290])],                      1, 24,  4, 256, "bf16"),
    ([(21, [1344 + i for i in range(9)])],                                   13, 15,  5, 128, "f16"),
    ([(30, [1920, 2100, 3000]), (0, [900]), (9, [600, 610]), (0, []), (40, [2600] * 11)], 7, 12, 4, 256, "bf16"),
    ([(33, [2150, 2200])],                                                   64, 12,  2, 128, "bf16"),
    ([(16, [1100, 1090, 1080])],                                             22, 24,  4, 256, "bf16"),
    ([(50, [3200 + 3 * i for i in range(40)])],                               1,  6,  1, 256, "f16"),
    ([(12, [800, 850, 900, 820])],                                            2, 128, 1, 128, "f16"),
    ([(70, [4490, 4480 + 63])],                                              64,  8,  8, 128, "bf16"),
    ([(24, [1536 + i for i in range(8)]) for _ in range(6)],                  1, 24,  4, 256, "bf16"),
    ([(100, [6400, 9000, 6500])],                                             4,  3,  3, 256, "bf16"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("out", ["f32", "same"])
def test_matches_the_formula(cuda_dev, i, out):
    s = make(*CASES[i], tree="chain" if i % 3 == 0 else "random", seed=i)
    check(s, torch.float32 if out == "f32" else s["q"].dtype)


def test_drawn_batches(cuda_dev):
    rng = np.random.default_rng(12)
    for seed in range(25):
        groups = []
        for _ in range(rng.integers(1, 7)):
            both = int(rng.integers(0, 30))
            groups.append((both, [int(both * PAGE + rng.integers(0, 400)) for _ in range(rng.integers(1, 9))]))
        Hkv = int(rng.integers(1, 5))
        s = make(groups, int(rng.integers(1, 30)), Hkv * int(rng.integers(1, 9)), Hkv, int(rng.choice([128, 256])),
                 str(rng.choice(["bf16", "f16"])), seed=seed)
        check(s, s["q"].dtype if seed % 2 else torch.float32)


def test_groups_do_not_change_results(cuda_dev):
    """The same batch as one group, as groups of one, and as pairs."""
    s = make([(30, [1930, 2000, 1990, 2500])], 6, 8, 2, 128, "f16", seed=3)
    ref = reference(s)
    for start in ([0, 4], [0, 1, 2, 3, 4], [0, 2, 4], [0, 1, 4], [0, 0, 4, 4]):
        s["group_start"] = torch.tensor(start, dtype=torch.int32)
        out, lse, status = call(s, torch.float32)
        assert status == 0
        near(out, lse, ref)


def test_scale_of_any_sign_and_no_lse(cuda_dev):
    s = make([(6, [400, 450])], 9, 4, 2, 128, "bf16", seed=5)
    for scale in (0.0, -0.05, 0.3):
        check(s, torch.float32, scale=scale)
    check(s, torch.bfloat16, lse=False)


def test_growing_scores_move_the_shift(cuda_dev):
    s = make([(20, [1300, 1400, 1350])], 10, 4, 1, 128, "bf16", seed=9, junk=0.0)
    s["q"] = torch.full_like(s["q"], 0.25)
    for b in range(3):
        for p in range(0 if b == 0 else 1280, int(s["ctx_len"][b])):
            at = int(s["page_table"][b, p // PAGE]), slice(None), p % PAGE
            s["k_pool"][at] = s["k_pool"][at] * 0.1 + p / 100
    check(s, torch.float32)
    check(s, torch.bfloat16)


def test_steep_scores(cuda_dev):
    """Scores that rise and fall by more than the exponent's range from one tile to the next."""
    s = make([(16, [1024, 1100, 1050])], 4, 4, 1, 128, "f16", seed=2, junk=0.0)
    for j in range(16):
        s["k_pool"][int(s["page_table"][0, j])] *= 40.0 if j % 4 == 1 else 0.01
    check(s, torch.float32, scale=1.0)


def test_tree_nodes_that_are_not_finite_stay_with_their_descendants(cuda_dev):
    LT = _lt()
    s = make([(10, [700, 650])], 12, 4, 2, 128, "bf16", seed=7)
    ref = reference(s)
    for name in ("k_tree", "v_tree"):
        t = dict(s)
        t[name] = s[name].clone()
        t[name][1, 5] = float("inf") if name == "v_tree" else float("nan")
        out, lse, status = call(t, torch.float32)
        sees = s["sees"][1, :, 5]
        good = torch.ones(2, 12, dtype=torch.bool)
        good[1] = ~sees
        near(out, lse, ref, good)
        assert status == LT.DEV_NONFINITE and torch.isnan(out[~good]).all() and torch.isnan(lse[~good]).all()


def test_rows_without_keys(cuda_dev):
    LT = _lt()
    s = make([(0, [0, 0]), (2, [130, 140])], 3, 4, 2, 128, "f16", seed=1)
    anc = s["anc_mask"].cuda().clone()
    anc[0, 1] = 0
    out, lse, status = call(s, torch.float32, anc=anc)
    assert status == LT.DEV_BAD_NODE
    assert (out[0, 1] == 0).all() and torch.isneginf(lse[0, 1]).all()
    good = torch.ones(4, 3, dtype=torch.bool)
    good[0, 1] = False
    near(out, lse, reference(s), good)


def test_pages_out_of_range_are_skipped(cuda_dev):
    LT = _lt()
    s = make([(20, [1300, 1290])], 3, 4, 2, 128, "f16", seed=4)
    pages = s["k_pool"].shape[0]
    table = s["page_table"].cuda()
    bad = table.clone()
    bad[0, 20] = pages + 5  # sequence 0's own
    out, lse, status = call(s, torch.float32, table=bad, plan_table=table)
    assert status == LT.DEV_BAD_PAGE
    ref = reference(s)
    near(out, lse, ref, [1])
    t = dict(s, ctx_len=torch.tensor([1280, 1290], dtype=torch.int32))
    near(out, lse, reference(t), [0])


def test_a_plan_of_other_sizes_writes_nothing(cuda_dev):
    LT = _lt()
    s = make([(20, [1300, 1290])], 3, 4, 2, 128, "f16", seed=4)
    d = {k: v.cuda() for k, v in s.items()}
    out = torch.full(s["q"].shape, 3.0, device="cuda")
    plan = torch.zeros(LT.lucetree_shared_plan_bytes(2, 3, 4, 2, 128, 1), dtype=torch.uint8, device="cuda")
    ws = torch.empty(LT.lucetree_verify_attn_shared_workspace(2, 3, 4, 2, 128, 1), dtype=torch.uint8, device="cuda")
    for N in (0, 4):
        status, shared = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        if N:
            plan = torch.zeros(LT.lucetree_shared_plan_bytes(2, N, 4, 2, 128, 1), dtype=torch.uint8, device="cuda")
            LT.lucetree_shared_plan(d["page_table"], d["ctx_len"], d["group_start"], N, 4, 2, 128, s["k_pool"].shape[0],
                                    shared, plan, status)
        LT.lucetree_verify_attn_shared(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"],
                                       d["v_tree"], d["anc_mask"], 1, plan, out, status, ws)
        torch.cuda.synchronize()
        assert int(status.item()) == LT.DEV_BAD_ROW and (out == 3).all()


def test_captured_on_another_stream_and_two_calls_at_once(cuda_dev):
    LT = _lt()
    cases = [make([(30, [1930, 2000, 1990, 2500])], 6, 8, 2, 128, "f16", seed=3),
             make([(25, [1700, 1650]), (3, [200, 300])], 6, 8, 2, 128, "f16", seed=8)]
    want = [call(s, torch.float16) for s in cases]
    side = [torch.cuda.Stream() for _ in cases]
    for s, w, st in zip(cases, want, side):
        st.wait_stream(torch.cuda.current_stream())
        out, lse, status = call(s, torch.float16, stream=st)
        assert status == 0 and torch.equal(out, w[0]) and torch.equal(lse, w[1])
    # two calls of their own plans and workspaces, captured, replayed at the same time
    runs = []
    for s, st in zip(cases, side):
        d = {k: v.cuda() for k, v in s.items()}
        (B, N, Hq, D), Hkv, groups = s["q"].shape, 2, s["group_start"].numel() - 1
        r = dict(out=torch.empty_like(d["q"]), status=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 shared=torch.empty(groups, dtype=torch.int32, device="cuda"), d=d,
                 plan=torch.empty(LT.lucetree_shared_plan_bytes(B, N, Hq, Hkv, D, groups), dtype=torch.uint8, device="cuda"),
                 ws=torch.empty(LT.lucetree_verify_attn_shared_workspace(B, N, Hq, Hkv, D, groups), dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            LT.lucetree_shared_plan(d["page_table"], d["ctx_len"], d["group_start"], N, Hq, Hkv, D, d["k_pool"].shape[0],
                                    r["shared"], r["plan"], r["status"])
            for _ in range(2):  # two layers of one step
                LT.lucetree_verify_attn_shared(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"],
                                               d["v_tree"], d["anc_mask"], groups, r["plan"], r["out"], r["status"], r["ws"])
        runs.append((graph, r))
    for _ in range(5):
        for (graph, r), st in zip(runs, side):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for (_, r), w in zip(runs, want):
        assert int(r["status"].item()) == 0 and torch.equal(r["out"].cpu(), w[0])


def test_repeated_calls_are_identical(cuda_dev):
    s = make([(50, [3200 + 3 * i for i in range(20)]), (0, [5000])], 3, 24, 4, 256, "bf16", seed=6)
    first = call(s, torch.bfloat16)
    for _ in range(4):
        again = call(s, torch.bfloat16)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_more_sequences_than_a_block_of_the_plan(cuda_dev):
    rng = np.random.default_rng(8)
    groups = [(int(x), [int(x) * PAGE + int(y) for y in rng.integers(0, 200, 6)]) for x in rng.integers(0, 9, 100)]
    check(make(groups, 1, 2, 1, 128, "bf16", seed=3), torch.bfloat16)


def test_pools_past_four_gigabytes(cuda_dev):
    s = make([(12, [800, 850, 790])], 5, 8, 4, 256, "bf16", seed=12, junk=0.0)
    ref = reference(s, p_step=P_STEP[torch.bfloat16])
    used, far = s["k_pool"].shape[0], 40000  # 128 KB a page: offsets past 2^32
    big = dict(s, page_table=torch.where(s["page_table"] >= 0, s["page_table"] + far - used, -1).to(torch.int32))
    for name in ("k_pool", "v_pool"):
        pool = torch.zeros(far, *s[name].shape[1:], dtype=s[name].dtype, device="cuda")
        pool[far - used:] = s[name].cuda()
        big[name] = pool
    out, lse, status = call(big, torch.bfloat16)
    assert status == 0
    near(out, lse, ref)


# groups of more than 128 rows, which pairs of CTAs take together
PAIRED = [([(10, [700, 650, 641, 720])], 12, 8, 2, 128, "bf16"), ([(10, [700, 650, 641, 720])], 12, 8, 2, 256, "f16"),
          ([(7, [460, 470]), (0, [300]), (3, [200] * 9)], 16, 12, 2, 256, "bf16")]


@pytest.mark.parametrize("i", range(len(PAIRED)))
@pytest.mark.parametrize("out", ["f32", "same"])
def test_pairs_and_nodes_that_are_not_finite(cuda_dev, i, out):
    """Values that are not finite in one half of the dims, or of the keys, reach the rows of both CTAs that see them."""
    LT = _lt()
    s = make(*PAIRED[i], seed=20 + i)
    t = s["q"].dtype if out == "same" else torch.float32
    ref = reference(s, p_step=P_STEP[t])
    out_, lse, status = call(s, t)
    assert status == 0
    near(out_, lse, ref)
    B, N, D = s["q"].shape[0], s["q"].shape[1], s["q"].shape[3]
    for b, node, dim, name in ((0, 3, 1, "v_tree"), (1, N - 1, D - 1, "v_tree"), (B - 1, 0, D // 2, "v_tree"), (1, 2, 5, "k_tree")):
        x = dict(s)
        x[name] = s[name].clone()
        x[name][b, node, 0, dim] = float("inf") if name == "v_tree" else float("nan")
        got, lse, status = call(x, t)
        assert status == LT.DEV_NONFINITE
        Hq, Hkv = s["q"].shape[2], s["k_tree"].shape[2]
        good = torch.ones(B, N, Hq, dtype=torch.bool)
        good[b, :, :Hq // Hkv] = ~s["sees"][b, :, node][:, None]  # (query heads of KV head 0)
        near(got, lse, ref, good)
        assert bool(torch.isnan(got[~good]).all()) and bool(torch.isnan(lse[~good]).all())


def test_pairs_rows_without_keys_and_missing_pages(cuda_dev):
    LT = _lt()
    s = make([(0, [0, 0, 0]), (4, [260, 300, 280])], 16, 8, 2, 128, "f16", seed=3)
    anc = s["anc_mask"].cuda().clone()
    anc[1, 9] = 0
    out, lse, status = call(s, torch.float32, anc=anc)
    assert status == LT.DEV_BAD_NODE
    assert bool((out[1, 9] == 0).all()) and bool(torch.isneginf(lse[1, 9]).all())
    good = torch.ones(6, 16, dtype=torch.bool)
    good[1, 9] = False
    near(out, lse, reference(s), good)
    table = s["page_table"].cuda()
    bad = table.clone()
    bad[4, 4] = -1  # positions 256 .. of sequence 4
    out, lse, status = call(s, torch.float32, table=bad, plan_table=table)
    assert status == LT.DEV_BAD_PAGE
    t = dict(s, ctx_len=torch.tensor([0, 0, 0, 260, 256, 280], dtype=torch.int32))
    near(out, lse, reference(t))


def test_pairs_growing_and_steep_scores(cuda_dev):
    s = make([(20, [1300, 1400, 1350])], 24, 4, 1, 256, "bf16", seed=9, junk=0.0)
    s["q"] = torch.full_like(s["q"], 0.25)
    for b in range(3):
        for p in range(0 if b == 0 else 1280, int(s["ctx_len"][b])):
            at = int(s["page_table"][b, p // PAGE]), slice(None), p % PAGE
            s["k_pool"][at] = s["k_pool"][at] * 0.1 + p / 100
    check(s, torch.float32)
    check(s, torch.bfloat16)
    s = make([(16, [1024, 1100, 1050])], 20, 4, 1, 128, "f16", seed=2, junk=0.0)
    for j in range(16):
        s["k_pool"][int(s["page_table"][0, j])] *= 40.0 if j % 4 == 1 else 0.01
    check(s, torch.float32, scale=1.0)


def test_pairs_are_identical_from_call_to_call(cuda_dev):
    for D, t in ((256, "bf16"), (128, "f16")):
        s = make([(40, [2600 + i for i in range(9)]), (0, [5000]), (33, [2200, 2300])], 22, 12, 2, D, t, seed=6)
        first = call(s, s["q"].dtype)
        for _ in range(4):
            again = call(s, s["q"].dtype)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_forked_prompt_decodes_with_shared_pages(cuda_dev):
    """A prompt appended, forked into beams, and decoded for some steps: rotation, plan, attention of two layers and
    commit on the library's calls, against a cache kept token by token."""
    LT = _lt()
    B, N, Hq, Hkv, D, layers, prompt = 6, 3, 8, 2, 128, 2, 200
    g, maxp, pages = torch.Generator().manual_seed(1), 8, 60
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    e = lambda *s, t=torch.int32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    steps, _ = LT.lucetree_rope_steps(64, 1e4)
    freq = 1e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    steps, status = steps.cuda(), i32(0)
    pools = [(r(pages, Hkv, PAGE, D), r(pages, Hkv, PAGE, D)) for _ in range(layers)]

    def turned(x, pos):  # x [n][H][D] at pos [n], as the cache holds it
        a = (pos[:, None].double() * freq)[:, None]
        x = x.double().cpu()
        y = x.clone()
        y[..., :32] = x[..., :32] * a.cos() - x[..., 32:64] * a.sin()
        y[..., 32:64] = x[..., :32] * a.sin() + x[..., 32:64] * a.cos()
        return y.to(torch.bfloat16).double()

    # the prompt
    table = torch.full((1, maxp), -1, dtype=torch.int32, device="cuda")
    table[0, :4] = i32(40, 3, 17, 5)
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    ref[table[0, :4].long()] = 1
    cache = []
    for k_pool, v_pool in pools:
        k, v = r(prompt, Hkv, D), r(prompt, Hkv, D)
        ctx = e(1)
        LT.lucetree_append_kv(k, v, i32(0, prompt), table, i32(0), ctx, k_pool, v_pool, status, steps=steps)
        cache.append([(turned(k, torch.arange(prompt)), v.double().cpu()) for _ in range(B)])
    # six beams of it
    src, out_t, ctx_b, ref_b, cs, cd = i32(*[0] * B), e(B, maxp), e(B), e(pages), e(B), e(B)
    ws = e(LT.lucetree_reorder_pages_workspace(1, B, pages), t=torch.uint8)
    LT.lucetree_reorder_pages(table, ctx, src, 2 * N * 4, ref, out_t, ctx_b, ref_b, cs, cd, status, ws)
    for pool in pools:
        LT.lucetree_copy_pages(cs, cd, *pool, status)
    plan = e(LT.lucetree_shared_plan_bytes(B, N, Hq, Hkv, D, 1), t=torch.uint8)
    aws = e(LT.lucetree_verify_attn_shared_workspace(B, N, Hq, Hkv, D, 1), t=torch.uint8)
    shared, anc = e(1), e(B, N, t=torch.int64)
    for step in range(4):
        parent = i32(-1, 0, 0).expand(B, N).contiguous()  # two continuations of node 0
        LT.lucetree_build_anc_mask(parent, anc, status)
        LT.lucetree_shared_plan(out_t, ctx_b, i32(0, B), N, Hq, Hkv, D, pages, shared, plan, status)
        assert int(shared.item()) == prompt // PAGE
        take = torch.tensor([(b + step) % 3 for b in range(B)])  # 0: node 0; 1, 2: that child too
        acc = torch.full((B, N), -1, dtype=torch.int32)
        acc[:, 0] = 0
        acc[take > 0, 1] = take[take > 0].int()
        n_acc = 1 + (take > 0).int()
        L = ctx_b.cpu()
        new_ctx = e(B)
        for layer, (k_pool, v_pool) in enumerate(pools):
            qkv = r(B, N, (Hq + 2 * Hkv) * D)
            q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
            qr, kt, vt = e(*q.shape, t=q.dtype), e(*k.shape, t=q.dtype), e(*v.shape, t=q.dtype)
            LT.lucetree_rope(q, k, steps, 0, qr, kt, status, ctx_len=ctx_b, anc_mask=anc, v=v, v_out=vt)
            out = e(B, N, Hq, D, t=torch.float32)
            LT.lucetree_verify_attn_shared(qr, k_pool, v_pool, out_t, ctx_b, kt, vt, anc, 1, plan, out, status, aws)
            LT.lucetree_commit(kt, vt, acc.cuda(), n_acc.int().cuda(), out_t, ctx_b, new_ctx, k_pool, v_pool, status)
            for b in range(B):
                pos = torch.tensor([L[b], L[b] + 1, L[b] + 1])
                kb, vb = turned(k[b], pos), v[b].double().cpu()
                qb = turned(q[b], pos)
                kc, vc = cache[layer][b]
                for i in range(N):
                    path = [0] if i == 0 else [0, i]
                    K, V = torch.cat([kc, kb[path]]), torch.cat([vc, vb[path]])
                    for h in range(Hq):
                        x = K[:, h // 4] @ qb[i, h] * D ** -0.5
                        p = torch.softmax(x, 0)
                        want = p @ V[:, h // 4]
                        # P in fp16: 2^-11 of a term, and 2^-25 of the largest; 2^-12 for a rotated value that lies next
                        # to the border of two bf16 values, where 32 and 64 bits may round apart (2^-8 of one of a
                        # score's 128 products, D^-0.5 of which the score has, for few keys)
                        room = (2.0 ** -11 + 2.0 ** -12) * (p @ V[:, h // 4].abs()) + 2.0 ** -25 * V[:, h // 4].abs().sum(0)
                        assert bool(((out[b, i, h].double().cpu() - want).abs() <= room).all())
                keep = acc[b][:int(n_acc[b])].long()
                cache[layer][b] = (torch.cat([kc, kb[keep]]), torch.cat([vc, vb[keep]]))
        ctx_b = new_ctx
        assert int(status.item()) == 0 and torch.equal(ctx_b.cpu(), L + n_acc)


@pytest.mark.parametrize("case", [
    ([(10, [700, 650, 800])], 5, 4, 2, 128, "bf16"),             # one block of three sequences
    ([(10, [700, 650, 641, 720])], 12, 8, 2, 256, "f16"),        # pairs
    ([(6, [500, 450] * 20), (0, [300])], 1, 12, 2, 128, "f16"),  # forty sequences of one node, one alone
    ([(6, [500, 450] * 20)], 6, 4, 4, 256, "bf16"),
    ([(12, [1100] * 6)] * 40, 3, 8, 2, 128, "bf16"),            # several pieces to a CTA
    ([(12, [1100] * 6)] * 40, 3, 24, 2, 256, "bf16"),           # ... and to a pair
], ids=lambda c: "%d-%d-%d-%d-%s" % (len(c[0]), c[1], c[2] // c[3], c[4], c[5]))
@pytest.mark.parametrize("out", ["f32", "same"])
def test_committed_values_that_are_not_finite_stay_with_their_sequences(cuda_dev, case, out):
    LT = _lt()
    s = make(*case, seed=13)
    B, N, Hq, D = s["q"].shape
    Hkv = s["k_tree"].shape[2]
    t = torch.float32 if out == "f32" else s["q"].dtype
    ref = reference(s, p_step=P_STEP[t])
    for b, pos, dim in ((1, int(s["ctx_len"][1]) - 1, 0), (B - 1, int(s["ctx_len"][B - 1]) - 2, D - 1), (0, 70, D // 2)):
        for value in (float("nan"), float("inf")):
            x = dict(s, v_pool=s["v_pool"].clone())
            page = int(s["page_table"][b, pos // PAGE])
            x["v_pool"][page, 1, pos % PAGE, dim] = value
            got, lse, status = call(x, t)
            assert status == LT.DEV_NONFINITE
            with_it = torch.tensor([page in s["page_table"][c, :-(-int(s["ctx_len"][c]) // PAGE)].tolist() for c in range(B)])
            good = torch.ones(B, N, Hq, dtype=torch.bool)
            good[with_it, :, Hq // Hkv:2 * (Hq // Hkv)] = False
            near(got, lse, ref, good)
            assert not bool(torch.isfinite(got[~good][:, dim]).any())


@pytest.mark.parametrize("case", [([(10, [700, 650, 800])], 5, 4, 2, 128, "bf16"),
                                  ([(10, [700, 650, 641, 720])], 12, 8, 2, 256, "f16")], ids=["one", "pair"])
def test_queries_and_committed_keys_that_are_not_finite_stay_with_their_rows(cuda_dev, case):
    LT = _lt()
    s = make(*case, seed=14)
    B, N, Hq, D = s["q"].shape
    G = Hq // s["k_tree"].shape[2]
    ref = reference(s)
    x = dict(s, q=s["q"].clone())
    x["q"][1, 2, G, 3] = float("nan")
    got, lse, status = call(x, torch.float32)
    good = torch.ones(B, N, Hq, dtype=torch.bool)
    good[1, 2, G] = False
    near(got, lse, ref, good)
    assert status == LT.DEV_NONFINITE and bool(torch.isnan(got[~good]).all()) and bool(torch.isnan(lse[~good]).all())
    x = dict(s, k_pool=s["k_pool"].clone())
    pos = int(s["ctx_len"][2]) - 1
    x["k_pool"][int(s["page_table"][2, pos // PAGE]), 0, pos % PAGE, D - 1] = float("nan")
    got, lse, status = call(x, torch.float32)
    good = torch.ones(B, N, Hq, dtype=torch.bool)
    good[2, :, :G] = False
    near(got, lse, ref, good)
    assert status == LT.DEV_NONFINITE and bool(torch.isnan(got[~good]).all()) and bool(torch.isnan(lse[~good]).all())


def test_a_broken_sequence_in_a_captured_call(cuda_dev):
    """A captured call with values that are not finite, replayed once they are mended."""
    LT = _lt()
    s = make([(10, [700, 650, 641, 720])], 12, 8, 2, 256, "bf16", seed=15)
    ref = reference(s)
    d = {k: v.cuda() for k, v in s.items()}
    B, N, Hq, D = s["q"].shape
    out, lse = torch.empty(B, N, Hq, D, device="cuda"), torch.empty(B, N, Hq, device="cuda")
    status, shared = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    plan = torch.empty(LT.lucetree_shared_plan_bytes(B, N, Hq, 2, D, 1), dtype=torch.uint8, device="cuda")
    ws = torch.empty(LT.lucetree_verify_attn_shared_workspace(B, N, Hq, 2, D, 1), dtype=torch.uint8, device="cuda")

    def run():
        LT.lucetree_shared_plan(d["page_table"], d["ctx_len"], d["group_start"], N, Hq, 2, D, d["k_pool"].shape[0], shared,
                                plan, status)
        LT.lucetree_verify_attn_shared(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"],
                                       d["v_tree"], d["anc_mask"], 1, plan, out, status, ws, lse=lse)

    page, slot = int(s["page_table"][3, 718 // PAGE]), 718 % PAGE
    was = d["v_pool"][page, 0, slot].clone()
    d["v_pool"][page, 0, slot] = float("nan")
    run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    good = torch.ones(B, N, Hq, dtype=torch.bool)
    good[3, :, :4] = False
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        near(out.cpu(), lse.cpu(), ref, good)
        assert bool(torch.isnan(out.cpu()[~good]).all())
    d["v_pool"][page, 0, slot] = was
    status.zero_()
    graph.replay()
    torch.cuda.synchronize()
    near(out.cpu(), lse.cpu(), ref)
    assert int(status.item()) == 0
