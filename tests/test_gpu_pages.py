"""Page tables, counts and copies: lucetree_reorder_pages, lucetree_trim_pages,
lucetree_compact_pages, lucetree_copy_pages and lucetree_reorder_states against
plain loops over rows and pages, and a run of them around windowed verify steps
and a beam selection."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 64


def _lt():
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    return LT


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _new(*shape):
    return torch.full(shape, -77, dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def draw_pool(rng, rows, P, spare, lengths=None, share=0.4, trim=0.2, extra=2):
    """Tables whose rows share some whole pages and own the others; some whole
    pages unmapped, some rows with entries past their length."""
    L = np.array([int(rng.integers(0, P * PAGE + 1)) for _ in range(rows)] if lengths is None else lengths)
    table, nxt = np.full((rows, P), -1), 0
    for b in range(rows):
        for c in range(min(P, -(-int(L[b]) // PAGE) + int(rng.integers(0, extra + 1)))):
            donor = int(rng.integers(0, b)) if b else 0
            if b and c < L[b] // PAGE and c < L[donor] // PAGE and rng.random() < share and table[donor, c] >= 0:
                table[b, c] = table[donor, c]
            elif c < L[b] // PAGE and rng.random() < trim:
                continue
            else:
                table[b, c] = nxt
                nxt += 1
    pages = nxt + spare
    ids = rng.permutation(pages)
    table = np.where(table >= 0, ids[np.clip(table, 0, None)], -1)
    ref = np.zeros(pages, int)
    np.add.at(ref, table[table >= 0], 1)
    return table, L, ref


def ref_reorder(table, L, ref, src, reserve):
    P, rows = table.shape[1], len(src)
    held, new = ref.copy(), ref.copy()
    free = list(np.nonzero(ref == 0)[0])
    out, ctx, cs, cd = np.full((rows, P), -1), np.zeros(rows, int), np.full(rows, -1), np.full(rows, -1)
    for b in range(table.shape[0]):
        for p in table[b][table[b] >= 0]:
            new[p] -= 1
    seen, short = set(), False
    for r, b in enumerate(src):
        if b < 0:
            continue
        ctx[r], full = L[b], L[b] // PAGE
        for c in range(min(P, -(-(int(L[b]) + reserve) // PAGE))):
            p = table[b, c]
            if c >= full and not (p >= 0 and held[p] == 1 and b not in seen):
                q = free.pop(0) if free else -1
                short |= q < 0
                if c == full and L[b] % PAGE and p >= 0 and q >= 0:
                    cs[r], cd[r] = p, q
                p = q
            out[r, c] = p
            if p >= 0:
                new[p] += 1
        seen.add(b)
    return out, ctx, new, cs, cd, short


def run_reorder(table, L, ref, src, reserve, in_place=False):
    LT = _lt()
    t, c, s, f = _dev(table), _dev(L), _dev(src), _dev(ref)
    rows, P = len(src), table.shape[1]
    out, ctx, cs, cd, st = _new(rows, P), _new(rows), _new(rows), _new(rows), _status()
    f_out = f if in_place else _new(len(ref))
    ws = torch.empty(LT.lucetree_reorder_pages_workspace(len(L), rows, len(ref)), dtype=torch.uint8, device="cuda")
    ws.fill_(0xEE)
    LT.lucetree_reorder_pages(t, c, s, reserve, f, out, ctx, f_out, cs, cd, st, ws)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (out, ctx, f_out, cs, cd)] + [int(st.item())]


@pytest.mark.parametrize("rows,rows_out,P,reserve,spare", [
    (1, 1, 1, 0, 4), (1, 4, 17, 22, 20), (3, 2, 5, 64, 9), (8, 8, 40, 1, 30), (8, 20, 9, 200, 120), (40, 64, 33, 22, 200),
    (5, 5, 1500, 8, 30), (2, 3, 70, 4032, 300), (1100, 1200, 3, 22, 2500), (6, 6, 12, 0, 9000),
    (30, 40, 700, 10, 300),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_reorder(cuda_dev, rows, rows_out, P, reserve, spare, in_place):
    rng = np.random.default_rng(rows * 1000 + P)
    L = rng.integers(0, max(1, P * PAGE - reserve) + 1, size=rows)
    table, L, ref = draw_pool(rng, rows, P, spare, np.minimum(L, max(0, P * PAGE - reserve)))
    src = rng.integers(-1, rows, size=rows_out)
    fits = (L + reserve <= P * PAGE).all()
    *got, status = run_reorder(table, L, ref, src, reserve, in_place)
    *want, short = ref_reorder(table, L, ref, src, reserve)
    assert not short
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert status == (0 if fits else _lt().DEV_BAD_CTX)


def test_reorder_when_the_pool_runs_out(cuda_dev):
    LT = _lt()
    rng = np.random.default_rng(7)
    table, L, ref = draw_pool(rng, 4, 8, 5, [130, 64, 0, 400])
    src = [0, 0, 0, 1, 1, 3, 3, 3, 2]
    *got, status = run_reorder(table, L, ref, src, 70)
    *want, short = ref_reorder(table, L, ref, np.array(src), 70)
    assert short and status == LT.DEV_NO_PAGE
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_reorder_tail_pages_held_by_two_rows_are_not_kept(cuda_dev):
    # both rows name the same partial page: neither may commit into it
    table, L = np.array([[3, 4, -1], [3, 4, -1]]), np.array([100, 100])
    ref = np.array([0, 0, 0, 2, 2, 0])
    *got, status = run_reorder(table, L, ref, [0, 1], 10)
    assert status == 0
    assert got[0].tolist() == [[3, 0, -1], [3, 1, -1]] and got[2].tolist() == [1, 1, 0, 2, 0, 0]
    assert got[3].tolist() == [4, 4] and got[4].tolist() == [0, 1]


def test_reorder_flags_bad_inputs_and_leaves_the_rest(cuda_dev):
    LT = _lt()
    table, L = np.array([[5, 6], [7, 99], [1, 2]]), np.array([70, 64, 1000])
    ref = np.array([0, 1, 1, 0, 0, 1, 1, 1])
    out, ctx, ref_out, cs, cd, status = run_reorder(table, L, ref, [0, 3, -2, 2, 1], 1)
    assert status == LT.DEV_BAD_ROW | LT.DEV_BAD_CTX | LT.DEV_BAD_PAGE
    assert out.tolist() == [[5, 6], [-1, -1], [-1, -1], [-1, -1], [7, 0]] and ctx.tolist() == [70, 0, 0, 0, 64]
    assert ref_out.tolist() == [1, 1, 1, 0, 0, 1, 1, 1]  # the row of unknown length keeps its pages
    assert (cs == -1).all() and (cd == -1).all()


def ref_trim(table, L, window, sinks, ref):
    table, ref = table.copy(), ref.copy()
    for b in range(table.shape[0]):
        for c in range(table.shape[1]):
            if c * PAGE >= sinks and (c + 1) * PAGE - 1 <= L[b] - window:
                if table[b, c] >= 0:
                    ref[table[b, c]] -= 1
                table[b, c] = -1
    return table, ref


@pytest.mark.parametrize("rows,P,window,sinks", [(1, 1, 1, 0), (3, 20, 100, 4), (7, 1100, 4096, 64), (5, 9, 64, 65),
                                                 (4, 30, 5000, 0), (300, 4, 1, 0), (40, 1100, 500, 4), (2, 6, 2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_trim(cuda_dev, rows, P, window, sinks, in_place):
    LT = _lt()
    rng = np.random.default_rng(rows + P)
    table, L, ref = draw_pool(rng, rows, P, 3)
    want = ref_trim(table, L, window, sinks, ref)
    t, c, f, st = _dev(table), _dev(L), _dev(ref), _status()
    t2, f2 = (t, f) if in_place else (_new(rows, P), _new(len(ref)))
    for _ in range(2 if in_place else 1):  # a second pass finds nothing more
        LT.lucetree_trim_pages(t, c, window, sinks, f, t2, f2, st)
    assert np.array_equal(t2.cpu().numpy(), want[0]) and np.array_equal(f2.cpu().numpy(), want[1])
    assert int(st.item()) == 0


def test_trim_flags(cuda_dev):
    LT = _lt()
    t, c, f, st = _dev([[0, 9, 2], [0, 1, 2]]), _dev([192, 500]), _dev([0, 1, 1]), _status()
    LT.lucetree_trim_pages(t, c, 1, 0, f, t, f, st)
    assert int(st.item()) == LT.DEV_BAD_CTX | LT.DEV_BAD_PAGE
    assert t.cpu().tolist() == [[-1, -1, -1], [0, 1, 2]] and f.cpu().tolist()[1:] == [1, 0]


def ref_compact(table, ref):
    live = int((ref > 0).sum())
    holes = [p for p in range(live) if ref[p] <= 0]
    movers = [p for p in range(live, len(ref)) if ref[p] > 0]
    name = dict(zip(movers, holes))
    new = ref.copy()
    for p, h in name.items():
        new[h], new[p] = ref[p], 0
    cs, cd = np.full(len(ref) // 2, -1), np.full(len(ref) // 2, -1)
    cs[:len(movers)], cd[:len(movers)] = movers, holes
    return np.vectorize(lambda p: name.get(int(p), int(p)))(table), new, cs, cd, len(movers), live


@pytest.mark.parametrize("rows,P,spare,used", [(1, 1, 0, 1.0), (1, 1, 1, 0.0), (3, 7, 5, 0.5), (20, 60, 3000, 0.3),
                                               (9, 40, 1024, 0.9), (2, 3, 5000, 0.5), (30, 90, 0, 0.6), (4, 600, 0, 1.0),
                                               (30, 90, 9000, 0.6), (60, 600, 100, 0.5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(cuda_dev, rows, P, spare, used, in_place):
    LT = _lt()
    rng = np.random.default_rng(rows * P + spare)
    table, L, ref = draw_pool(rng, rows, P, spare, extra=0) if P > 1 else \
        (np.array([[0 if used else -1]]), [1], np.array([1 if used else 0] + [0] * spare))
    for b in range(rows):  # give some entries back
        for c in range(P):
            if table[b, c] >= 0 and rng.random() > used:
                ref[table[b, c]] -= 1
                table[b, c] = -1
    want = ref_compact(table, ref)
    n = len(ref)
    t, f, st = _dev(table), _dev(ref), _status()
    t2, f2 = (t, f) if in_place else (_new(rows, P), _new(n))
    cs, cd, cn, live = _new(n // 2), _new(n // 2), _new(1), _new(1)
    ws = torch.empty(LT.lucetree_compact_pages_workspace(n), dtype=torch.uint8, device="cuda")
    ws.fill_(0xEE)
    LT.lucetree_compact_pages(t, f, t2, f2, cs, cd, cn, live, st, ws)
    for g, w in zip((t2, f2, cs, cd), want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert int(cn.item()) == want[4] and int(live.item()) == want[5] and int(st.item()) == 0


def test_compact_flags_entries_that_name_no_page(cuda_dev):
    LT = _lt()
    t, f, st = _dev([[5, 3, 9, -4]]), _dev([0, 0, 0, 1, 0, 0]), _status()
    cs, cd, cn, live = _new(3), _new(3), _new(1), _new(1)
    ws = torch.empty(LT.lucetree_compact_pages_workspace(6), dtype=torch.uint8, device="cuda")
    LT.lucetree_compact_pages(t, f, t, f, cs, cd, cn, live, st, ws)
    assert t.cpu().tolist() == [[-1, 0, -1, -1]] and f.cpu().tolist() == [1, 0, 0, 0, 0, 0]
    assert int(st.item()) == LT.DEV_BAD_PAGE


@pytest.mark.parametrize("shape,shape_v", [((3, 64, 128), (3, 64, 128)), ((1, 64, 8), (1, 64)), ((2, 64, 1000), None),
                                           ((4, 64, 256), (4, 64, 128))])
def test_copy_pages(cuda_dev, shape, shape_v):
    LT = _lt()
    rng = np.random.default_rng(1)
    pages = 60
    ids = rng.permutation(pages)
    src, dst = ids[:25].copy(), ids[25:50].copy()
    src[[3, 9]] = dst[[3, 9]] = -1
    src[5] = src[4]                                    # one page to two places
    pool = torch.from_numpy(rng.integers(-128, 127, size=(pages, *shape), dtype=np.int8)).cuda()
    v = None if shape_v is None else torch.from_numpy(rng.integers(-99, 99, size=(pages, *shape_v), dtype=np.int16)).cuda()
    for count in (None, 7, 0, 100, -5):
        k2, v2 = pool.clone(), None if v is None else v.clone()
        cnt = None if count is None else _dev([count])
        st = _status()
        LT.lucetree_copy_pages(_dev(src), _dev(dst), k2, v2, st, count=cnt)
        n = len(src) if count is None else max(0, min(len(src), count))
        for got, was in ((k2, pool), (v2, v)):
            if got is None:
                continue
            want = was.clone()
            for i in range(n):
                if src[i] >= 0:
                    want[int(dst[i])] = was[int(src[i])]
            assert torch.equal(got, want)
        assert int(st.item()) == 0


def test_copy_pages_past_four_gigabytes_and_bad_pages(cuda_dev):
    LT = _lt()
    pages = 40000                                      # 5.2 GB
    pool = torch.zeros(pages, 4, 64, 256, dtype=torch.bfloat16, device="cuda")
    pool[39999] = 3.0
    pool[2] = 5.0
    st = _status()
    LT.lucetree_copy_pages(_dev([39999, 2]), _dev([0, 39998]), pool, None, st)
    assert int(st.item()) == 0 and (pool[0] == 3).all() and (pool[39998] == 5).all() and (pool[39997] == 0).all()
    before = float(pool[1].sum())
    LT.lucetree_copy_pages(_dev([40000, -1, 2, -2]), _dev([1, 1, -1, -2]), pool, None, st)
    assert int(st.item()) == LT.DEV_BAD_PAGE and float(pool[1].sum()) == before


@pytest.mark.parametrize("rows,rows_out,shape", [(1, 1, (4,)), (3, 7, (2, 128, 128)), (9, 4, (5, 12)), (2, 300, (4096,))])
def test_reorder_states(cuda_dev, rows, rows_out, shape):
    LT = _lt()
    rng = np.random.default_rng(rows)
    x = torch.randn(rows, *shape, device="cuda")
    src = rng.integers(-1, rows, size=rows_out)
    out = torch.full((rows_out, *shape), 9.0, device="cuda")
    st = _status()
    LT.lucetree_reorder_states(x, _dev(src), out, st)
    for r, b in enumerate(src):
        assert torch.equal(out[r], x[int(b)] if b >= 0 else torch.full_like(x[0], 9.0))
    assert int(st.item()) == 0
    LT.lucetree_reorder_states(x, _dev([rows] + [-1] * (rows_out - 1)), out, st)
    assert int(st.item()) == LT.DEV_BAD_ROW


def test_captured_and_replayed(cuda_dev):
    LT = _lt()
    rng = np.random.default_rng(17)
    table, L, ref = draw_pool(rng, 6, 20, 40, rng.integers(0, 1200, size=6), extra=0)
    pools = torch.randn(len(ref), 2, PAGE, 8, generator=torch.Generator().manual_seed(1)).cuda()
    t, c, f, src, st = _dev(table), _dev(L), _dev(ref), _dev([0] * 6), _status()
    k, v = pools.clone(), pools.clone()
    out, ctx, f2, cs, cd = _new(6, 20), _new(6), _new(len(ref)), _new(6), _new(6)
    ms, md, mn, live = _new(len(ref) // 2), _new(len(ref) // 2), _new(1), _new(1)
    state, state2 = torch.randn(6, 8, device="cuda"), torch.zeros(6, 8, device="cuda")
    ws = torch.empty(max(LT.lucetree_reorder_pages_workspace(6, 6, len(ref)), LT.lucetree_compact_pages_workspace(len(ref))),
                     dtype=torch.uint8, device="cuda")

    def go():
        LT.lucetree_reorder_pages(t, c, src, 9, f, out, ctx, f2, cs, cd, st, ws)
        LT.lucetree_copy_pages(cs, cd, k, v, st)
        LT.lucetree_reorder_states(state, src, state2, st)
        LT.lucetree_trim_pages(out, ctx, 200, 4, f2, out, f2, st)
        LT.lucetree_compact_pages(out, f2, out, f2, ms, md, mn, live, st, ws)
        LT.lucetree_copy_pages(ms, md, k, v, st, count=mn)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for pick in ([0, 0, 1, 5, -1, 3], [5, 4, 3, 2, 1, 0], [2, 2, 2, 2, 2, 2]):
        src.copy_(_dev(pick))
        k.copy_(pools)
        v.copy_(pools)
        graph.replay()
        torch.cuda.synchronize()
        o, cx, rf, a, b, short = ref_reorder(table, L, ref, np.array(pick), 9)
        want = pools.clone()
        for x, y in zip(a, b):
            if x >= 0:
                want[int(y)] = pools[int(x)]
        o, rf = ref_trim(o, cx, 200, 4, rf)
        o, rf, a, b, n, lv = ref_compact(o, rf)
        for x, y in zip(a[:n], b[:n]):
            want[int(y)] = want[int(x)]
        assert not short and np.array_equal(out.cpu().numpy(), o) and np.array_equal(f2.cpu().numpy(), rf)
        assert int(live.item()) == lv and torch.equal(k, want) and torch.equal(v, want)
        for r, x in enumerate(pick):
            assert x < 0 or torch.equal(state2[r], state[x])
    assert int(st.item()) == 0


def test_a_search_over_a_windowed_cache(cuda_dev):
    """Two requests: a prompt each, forked into beams by a selection, windowed
    attention and commits on the forks, a second selection that drops and
    doubles beams, pages behind the window given back and the pool closed up;
    attention reads the same keys all along."""
    LT = _lt()
    g = torch.Generator().manual_seed(5)
    B, K, V, Hq, Hkv, D, W, S, P = 2, 4, 777, 4, 2, 128, 150, 4, 12
    L0 = [333, 200]
    pages = 80
    dtype = torch.bfloat16
    perm = torch.randperm(pages, generator=g).tolist()
    table = np.full((B, P), -1)
    for b in range(B):
        for c in range(-(-(L0[b] + 2) // PAGE)):
            table[b, c] = perm.pop()
    ref = np.zeros(pages, int)
    ref[table[table >= 0]] = 1
    kp, vp = (torch.randn(pages, Hkv, PAGE, D, generator=g).to(dtype).cuda() for _ in range(2))
    # what each row's positions hold, kept apart from the pool
    hist = [[(kp[table[b, p // PAGE], :, p % PAGE].clone(), vp[table[b, p // PAGE], :, p % PAGE].clone())
             for p in range(L0[b])] for b in range(B)]
    table, ctx, ref, st = _dev(table), _dev(L0), _dev(ref), _status()
    states = torch.randn(B, 3, 16, generator=g).cuda()
    held = [states[b].clone() for b in range(B)]
    cum = torch.zeros(B, 1)
    moved = dropped = 0
    for step in range(4):
        rows, beams = table.shape[0], table.shape[0] // B
        logits = 2 * torch.randn(B, beams, V, generator=g)
        score, token, row, fin = torch.empty(B, K, device="cuda"), _new(B, K), _new(B, K), _new(B, K)
        ws = torch.empty(LT.lucetree_beam_select_workspace(B, beams, K, V), dtype=torch.uint8, device="cuda")
        LT.lucetree_beam_select(logits.cuda(), cum.cuda(), None, -1, score, token, row, fin, ws)
        cum = score.cpu()
        src = row.view(-1)
        new_t, new_c, cs, cd = _new(B * K, P), _new(B * K), _new(B * K), _new(B * K)
        ws = torch.empty(LT.lucetree_reorder_pages_workspace(rows, B * K, pages), dtype=torch.uint8, device="cuda")
        LT.lucetree_reorder_pages(table, ctx, src, 2, ref, new_t, new_c, ref, cs, cd, st, ws)
        LT.lucetree_copy_pages(cs, cd, kp, vp, st)
        new_s = torch.empty(B * K, 3, 16, device="cuda")
        LT.lucetree_reorder_states(states, src, new_s, st)
        hist = [list(hist[b]) for b in src.tolist()]
        held = [held[b] for b in src.tolist()]
        table, ctx, states = new_t, new_c, new_s
        # one token each: attend, then commit it
        R = B * K
        q, kt, vt = (torch.randn(R, 1, h, D, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
        out = torch.empty(R, 1, Hq, D, device="cuda")
        ws = torch.empty(LT.lucetree_verify_attn_workspace(R, 1, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        anc = torch.ones(R, 1, dtype=torch.int64, device="cuda")
        LT.lucetree_verify_attn_win(q, kp, vp, table, ctx, kt, vt, anc, W, S, out, st, ws)
        for r in range(R):
            n = len(hist[r])
            seen = [hist[r][p] for p in range(n) if p < S or n - p < W] + [(kt[r, 0], vt[r, 0])]
            k, v = (torch.stack([e[i] for e in seen]).double() for i in (0, 1))
            for h in range(Hq):
                x = k[:, h // 2] @ q[r, 0, h].double() * D ** -0.5
                p = torch.softmax(x, 0)
                want = p @ v[:, h // 2]
                # fp16 P (half a step), fp32 scores of D products, small terms flushed
                err = D * 2.0 ** -24 * float((k[:, h // 2].abs() @ q[r, 0, h].double().abs()).max()) * D ** -0.5
                tol = (2.0 ** -11 + 2 * err + 2.0 ** -20) * (p @ v[:, h // 2].abs()) + \
                    2.0 ** -25 * float(p.max()) * v[:, h // 2].abs().sum(0)
                assert ((out[r, 0, h].double() - want).abs() <= tol + 2.0 ** -24 * want.abs()).all()
            hist[r].append((kt[r, 0].clone(), vt[r, 0].clone()))
            assert torch.equal(states[r], held[r])
        acc, alen = torch.zeros(R, 1, dtype=torch.int32, device="cuda"), torch.ones(R, dtype=torch.int32, device="cuda")
        LT.lucetree_commit(kt, vt, acc, alen, table, ctx, ctx, kp, vp, st)
        before = int((ref > 0).sum())
        LT.lucetree_trim_pages(table, ctx, W, S, ref, table, ref, st)
        dropped += before - int((ref > 0).sum())
        cs, cd, cn, live = _new(pages // 2), _new(pages // 2), _new(1), _new(1)
        ws = torch.empty(LT.lucetree_compact_pages_workspace(pages), dtype=torch.uint8, device="cuda")
        LT.lucetree_compact_pages(table, ref, table, ref, cs, cd, cn, live, st, ws)
        LT.lucetree_copy_pages(cs, cd, kp, vp, st, count=cn)
        moved += int(cn.item())
        gone = int(live.item())
        assert int((ref > 0).sum()) == gone and int((ref[:gone] > 0).sum()) == gone
        kp[gone:] = float("nan")                       # nothing past the live pages is read again
        vp[gone:] = float("nan")
        counts = torch.bincount(table[table >= 0].long(), minlength=pages)
        assert torch.equal(counts.int(), ref)
    assert int(st.item()) == 0 and moved > 0 and dropped > 0
