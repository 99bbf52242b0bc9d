"""Tree-verify attention with a sliding window and sinks against the formula in
64 bits: windows from one position to past the context, sinks inside, at and
past page edges, sequences of length zero and one, deep chains that outgrow the
window, and anything at all in the positions that no node sees."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _lt():
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    return LT


def make(ctx, N, Hq, Hkv, D, dtype, window, sinks, tree="random", seed=0, spare=3):
    """Inputs with NaN wherever no node may look and -1 for pages it need not have."""
    rng = np.random.default_rng(seed)
    t = TYPES[dtype]
    B = len(ctx)
    per = [-(-(L + N) // PAGE) for L in ctx]
    pages = sum(per) + spare
    ids = rng.permutation(pages)
    table = np.full((B, max(per)), -1, np.int32)
    g = torch.Generator().manual_seed(seed)
    pools = [torch.full((pages, Hkv, PAGE, D), float("nan"), dtype=t) for _ in range(2)]
    at = 0
    for b, L in enumerate(ctx):
        table[b, :per[b]] = ids[at:at + per[b]]
        at += per[b]
        lo = max(0, L - window + 1)
        for p in range(L):
            if p < sinks or p >= lo:
                for pool in pools:
                    pool[table[b, p // PAGE], :, p % PAGE] = torch.randn(Hkv, D, generator=g).to(t)
        for c in range(per[b]):
            if c * PAGE >= sinks and (c + 1) * PAGE <= lo:
                table[b, c] = -1
    parent = np.full((B, N), -1, np.int64)
    for i in range(1, N):
        parent[:, i] = i - 1 if tree == "chain" else rng.integers(-1, i, size=B)
    paths = []
    for b in range(B):
        for i in range(N):
            path, c = [], i
            while c >= 0:
                path.append(c)
                c = parent[b, c]
            paths.append(path[::-1])
    anc = np.zeros((B, N), np.uint64)
    for n, path in enumerate(paths):
        anc[n // N, n % N] = np.uint64(sum(1 << int(j) for j in path))
    r = lambda *s: torch.randn(*s, generator=g).to(t)  # noqa: E731
    return dict(q=r(B, N, Hq, D), k_pool=pools[0], v_pool=pools[1], page_table=torch.from_numpy(table),
                ctx_len=torch.tensor(ctx, dtype=torch.int32), k_tree=r(B, N, Hkv, D), v_tree=r(B, N, Hkv, D),
                anc_mask=torch.from_numpy(anc.view(np.int64)), paths=paths, window=window, sinks=sinks)


def reference(s, scale=None, p_step=2.0 ** -11):
    """(out, lse, bound): the formula in 64 bits, row by row, and how far a
    correct kernel's output may be from it.

    P is rounded to fp16 (half a step: 2^-11 of each term; with a bf16 output to
    bf16: 2^-8) relative to a shift that lies within the factor 2^8 of the row's
    largest term, so a term below 2^-24 of it is off by at most 2^-25.  A score is a sum of D exact products
    in fp32: off by at most D 2^-24 sum|q k| scale, which moves each term by
    that fraction; 2^-20 more covers the exponential, the sums and the shifts."""
    q, (B, N, Hq, D) = s["q"].double(), s["q"].shape
    Hkv = s["k_tree"].shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, lse = torch.zeros(B, N, Hq, D, dtype=torch.float64), torch.full((B, N, Hq), float("-inf"), dtype=torch.float64)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        L = int(s["ctx_len"][b])
        for i in range(N):
            path = s["paths"][b * N + i]
            t = L + len(path) - 1
            pos = [p for p in range(L) if p < s["sinks"] or t - p < s["window"]]
            tree = [j for d, j in enumerate(path) if L + d < s["sinks"] or t - (L + d) < s["window"]]
            page = [int(s["page_table"][b, p // PAGE]) for p in pos]
            slot = [p % PAGE for p in pos]
            for g in range(Hkv):
                k = torch.cat([s["k_pool"][page, g, slot], s["k_tree"][b, tree, g]]).double()
                v = torch.cat([s["v_pool"][page, g, slot], s["v_tree"][b, tree, g]]).double()
                hs = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
                x = q[b, i, hs] @ k.T * scale
                lse[b, i, hs] = torch.logsumexp(x, -1)
                p = torch.exp(x - lse[b, i, hs, None])
                out[b, i, hs] = p @ v
                err = (D * 2.0 ** -24 * abs(scale) * (q[b, i, hs].abs() @ k.abs().T)).amax(-1, keepdim=True) + 2.0 ** -20
                bound[b, i, hs] = (p_step + 2 * err) * (p @ v.abs()) + \
                    2.0 ** -25 * p.amax(-1, keepdim=True) * v.abs().sum(0)
                lse_bound[b, i, hs] = err[:, 0] + 2.0 ** -24 * lse[b, i, hs].abs()
    return out, lse, bound, lse_bound


P_STEP = {torch.float32: 2.0 ** -11, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def call(s, out_dtype, lse=True, scale=None, stream=None):
    LT = _lt()
    d = {k: v.cuda() for k, v in s.items() if torch.is_tensor(v)}
    B, N, Hq, D = s["q"].shape
    out = torch.full((B, N, Hq, D), float("nan"), dtype=out_dtype, device="cuda")
    lse_t = torch.full((B, N, Hq), float("nan"), device="cuda") if lse else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(LT.lucetree_verify_attn_workspace(B, N, Hq, s["k_tree"].shape[2], D), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0x7F)  # garbage (3.4e38 as fp32): a partial read before it is written shows
    LT.lucetree_verify_attn_win(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"],
                                d["v_tree"], d["anc_mask"], s["window"], s["sinks"], out, status, ws, lse=lse_t,
                                scale=scale, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), None if lse_t is None else lse_t.cpu(), int(status.item())


def check(s, out_dtype, **kw):
    out, lse, status = call(s, out_dtype, **kw)
    ref, ref_lse, bound, lse_bound = reference(s, kw.get("scale"), P_STEP[out_dtype])
    assert status == 0
    bound = bound + (0 if out_dtype == torch.float32 else torch.finfo(out_dtype).eps / 2) * (ref.abs() + bound)
    assert torch.isfinite(out).all()
    assert ((out.double() - ref).abs() <= bound + 2.0 ** -24 * ref.abs()).all(), \
        float(((out.double() - ref).abs() / bound).max())
    if lse is not None:
        assert ((lse.double() - ref_lse).abs() <= lse_bound).all()


#       ctx,                          N,  Hq, Hkv, D,  dtype,  window, sinks, tree
CASES = [
    ((1000,),                          8,  8,  2, 128, "f16",  256,   4, "random"),
    ((0, 1, 63, 64, 65, 127, 300),     3,  4,  2, 128, "bf16", 100,   0, "random"),
    ((0, 1, 63, 64, 65, 127, 300),     5,  2,  1, 256, "f16",  1,     0, "chain"),
    ((64, 128, 200),                   6,  6,  3, 128, "f16",  1,     4, "chain"),
    ((500, 129),                      64,  2,  1, 128, "bf16", 5,     0, "chain"),   # nodes outgrow the window
    ((500, 129, 20),                  64,  4,  2, 256, "bf16", 40,   70, "chain"),   # two sink pages
    ((900, 130),                      33,  3,  1, 256, "f16",  63,  130, "random"),  # three sink pages: odd
    ((400, 700),                       7,  6,  2, 256, "bf16", 5000,  4, "random"),  # wider than the context
    ((400, 100),                       7,  6,  2, 256, "bf16", 10, 5000, "random"),  # sinks past the context
    ((1500, 777, 778, 40),            13, 15,  5, 128, "f16",  777,  70, "random"),
    ((3000, 1200),                    22, 24,  4, 256, "bf16", 1024,  4, "random"),
    ((2500,),                         64, 12,  2, 128, "bf16", 600,   1, "random"),  # several row groups
    ((1111, 70),                       1, 24,  4, 256, "bf16", 512,   4, "chain"),   # single-token decode
    ((700,),                           2, 144, 1, 128, "f16",  300,  10, "chain"),   # many heads to one KV head
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"w{c[6]}-s{c[7]}-n{c[1]}-d{c[4]}-{c[5]}")
@pytest.mark.parametrize("out", ["f32", "same"])
def test_matches_the_formula(cuda_dev, case, out):
    *shape, window, sinks, tree = case
    s = make(*shape, window, sinks, tree, seed=len(case[0]) + window)
    check(s, torch.float32 if out == "f32" else s["q"].dtype)


@pytest.mark.parametrize("shift", range(0, 66, 5))
def test_every_alignment_of_the_window_edge(cuda_dev, shift):
    s = make((900 + shift, 513 + shift), 40, 2, 1, 128, "f16", 320, 64 + shift, "chain", seed=shift)
    check(s, torch.float32)


def test_scale_of_any_sign_and_no_lse(cuda_dev):
    s = make((300, 90), 9, 4, 2, 128, "bf16", 77, 3, "chain", seed=5)
    for scale in (0.0, -0.05, 0.3):
        check(s, torch.float32, scale=scale)
    check(s, torch.bfloat16, lse=False)


def test_growing_scores_move_the_shift(cuda_dev):
    # keys grow along the window, so the softmax's shift has to move in every tile
    s = make((1400,), 30, 4, 1, 128, "bf16", 1000, 4, "chain", seed=9)
    q = torch.full_like(s["q"], 0.25)
    s["q"] = q
    for p in range(401, 1400):
        s["k_pool"][int(s["page_table"][0, p // PAGE]), :, p % PAGE] *= 0.1
        s["k_pool"][int(s["page_table"][0, p // PAGE]), :, p % PAGE] += p / 200
    check(s, torch.float32)


def test_a_batch_larger_than_a_warp(cuda_dev):
    rng = np.random.default_rng(4)
    ctx = tuple(int(x) for x in rng.integers(0, 260, size=70))
    check(make(ctx, 2, 2, 1, 128, "f16", 90, 4, "chain", seed=1), torch.float16)


def test_more_sequences_than_the_merge_lists_at_once(cuda_dev):
    rng = np.random.default_rng(8)
    ctx = tuple(int(x) for x in rng.integers(0, 400, size=1100))
    check(make(ctx, 1, 2, 1, 128, "bf16", 150, 4, "chain", seed=3), torch.bfloat16)


def test_pages_past_four_gigabytes(cuda_dev):
    s = make((900, 300), 5, 8, 4, 256, "bf16", 200, 4, "random", seed=12)
    ref, _, bound, _ = reference(s, p_step=P_STEP[torch.bfloat16])
    LT = _lt()
    used = s["k_pool"].shape[0]
    pools = []
    for name in ("k_pool", "v_pool"):
        big = torch.empty(40000, 4, PAGE, 256, dtype=torch.bfloat16, device="cuda")  # 5.2 GB
        big[40000 - used:] = s[name].cuda()
        pools.append(big)
    table = torch.where(s["page_table"] >= 0, s["page_table"] + 40000 - used, s["page_table"]).to(torch.int32).cuda()
    d = {k: s[k].cuda() for k in ("q", "ctx_len", "k_tree", "v_tree", "anc_mask")}
    out, st = torch.empty_like(d["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(LT.lucetree_verify_attn_workspace(2, 5, 8, 4, 256), dtype=torch.uint8, device="cuda")
    LT.lucetree_verify_attn_win(d["q"], *pools, table, d["ctx_len"], d["k_tree"], d["v_tree"], d["anc_mask"], 200, 4, out,
                                st, ws)
    assert int(st.item()) == 0
    assert ((out.cpu().double() - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()


def test_pages_that_are_missing_are_left_out(cuda_dev):
    # every page of the first tiles is missing: the keys that remain give the answer
    s = make((1000,), 4, 4, 1, 128, "f16", 600, 0, "chain", seed=13)
    gone = (1000 - 600 + 1) // PAGE, (1000 - 600 + 1) // PAGE + 5
    s["page_table"][0, gone[0]:gone[1]] = -1
    out, _, status = call(s, torch.float32)
    assert status == _lt().DEV_BAD_PAGE
    # a node at depth d, at t = 1000 + d, sees p iff t - p < window: the first one left is p = 64 * gone[1], so
    # the same keys lie in a window of t - p + 1 positions
    for i in range(4):
        t = dict(s, window=1000 + i - gone[1] * PAGE + 1)
        ref, _, bound, _ = reference(t)
        assert ((out[0, i].double() - ref[0, i]).abs() <= bound[0, i] + 2.0 ** -24 * ref[0, i].abs()).all()


def test_two_calls_at_once(cuda_dev):
    LT = _lt()
    sets = [make((1500, 700, 90), 22, 12, 2, 128, "bf16", 400, 4, "random", seed=s) for s in (21, 22)]
    want = [reference(s, p_step=P_STEP[torch.bfloat16]) for s in sets]
    dev = [{k: v.cuda() for k, v in s.items() if torch.is_tensor(v)} for s in sets]
    outs = [torch.empty_like(d["q"]) for d in dev]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = [torch.empty(LT.lucetree_verify_attn_workspace(3, 22, 12, 2, 128), dtype=torch.uint8, device="cuda")
          for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(25):
        for i, d in enumerate(dev):
            LT.lucetree_verify_attn_win(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"],
                                        d["v_tree"], d["anc_mask"], 400, 4, outs[i], st, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for o, (ref, _, bound, _) in zip(outs, want):
        assert ((o.cpu().double() - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()


def test_wide_window_is_the_full_attention(cuda_dev):
    LT = _lt()
    s = make((700, 65, 1300), 22, 24, 4, 256, "bf16", 4000, 0, "random", seed=2)
    got, lse, status = call(s, torch.float32)
    d = {k: v.cuda() for k, v in s.items() if torch.is_tensor(v)}
    out, st = torch.empty(got.shape, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(LT.lucetree_verify_attn_workspace(3, 22, 24, 4, 256), dtype=torch.uint8, device="cuda")
    lse2 = torch.empty(lse.shape, device="cuda")
    LT.lucetree_verify_attn(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"], d["v_tree"],
                            d["anc_mask"], out, st, ws, lse=lse2)
    _, _, bound, lse_bound = reference(s)
    assert status == 0 and int(st.item()) == 0
    assert ((got.double() - out.cpu().double()).abs() <= 2 * bound).all()
    assert ((lse.double() - lse2.cpu().double()).abs() <= 2 * lse_bound).all()


def test_rows_that_see_nothing_and_bad_inputs_are_flagged(cuda_dev):
    LT = _lt()
    s = make((200, 300), 4, 4, 2, 128, "bf16", 1, 0, "chain", seed=3)
    s["anc_mask"][0, 2] = 0b0011  # lacks the node itself
    s["anc_mask"][1, 0] = 0
    out, lse, status = call(s, torch.float32)
    assert status == LT.DEV_BAD_NODE
    assert (out[1, 0] == 0).all() and torch.isneginf(lse[1, 0]).all() and torch.isfinite(out).all()
    s = make((200, 300), 4, 4, 2, 128, "bf16", 150, 4, "chain", seed=3)
    s["page_table"][1, 3] = 99
    assert call(s, torch.float32)[2] & LT.DEV_BAD_PAGE
    s = make((200, 300), 4, 4, 2, 128, "bf16", 150, 4, "chain", seed=3)
    s["ctx_len"][0] = -5
    assert call(s, torch.float32)[2] & LT.DEV_BAD_CTX


def test_captured_and_replayed_on_another_stream(cuda_dev):
    LT = _lt()
    a = make((1200, 333), 6, 8, 2, 128, "bf16", 200, 4, "random", seed=6)
    b = make((1200, 333), 6, 8, 2, 128, "bf16", 200, 4, "random", seed=7)
    names = ("q", "k_pool", "v_pool", "page_table", "ctx_len", "k_tree", "v_tree", "anc_mask")
    d = {k: a[k].cuda() for k in names}
    out, st = torch.empty(2, 6, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32,
                                                                                         device="cuda")
    ws = torch.empty(LT.lucetree_verify_attn_workspace(2, 6, 8, 2, 128), dtype=torch.uint8, device="cuda")
    go = lambda: LT.lucetree_verify_attn_win(*(d[k] for k in names), 200, 4, out, st, ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for s in (b, a):
        for k in names:
            d[k].copy_(s[k])
        out.fill_(float("nan"))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        torch.cuda.synchronize()
        ref, _, bound, _ = reference(s, p_step=P_STEP[out.dtype])
        assert ((out.cpu().double() - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 64), (2, 4), (60, 4), (63, 0), (130, 0), (190, 4), (260, 70)])
@pytest.mark.parametrize("ctx,N,Hq,Hkv,D", [((700, 0, 5, 1000), 8, 8, 2, 128), ((900, 333), 22, 24, 4, 256),
                                            ((400,) * 40, 3, 8, 4, 128), ((640, 77), 40, 6, 1, 128)])
def test_segments_of_a_few_tiles(cuda_dev, window, sinks, ctx, N, Hq, Hkv, D):
    """Few and many rows, one and several row groups, fewer and more segments than SMs, at the
    sizes where a segment is left to one CTA or cut."""
    s = make(ctx, N, Hq, Hkv, D, "bf16", window, sinks, "random", seed=window + sinks)
    check(s, torch.bfloat16)
