"""Cases and plain forms of the decoding-state operators: tree-verify attention
with a sliding window and sinks, beam selection, and the paged cache's
reorder / trim / compact / copy.

``own`` chooses what ``run`` computes: False, the plain form in elementary
torch operations; True, the library's calls on the same inputs.
"""
import random

import numpy as np
import torch

own = False

PAGE = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    win = dict(op="window", dtype="bf16", Hq=24, Hkv=4, D=256, chain=False, trimmed=True)
    beam = dict(op="beam", dtype="f32", V=151936, done=False, masked=False)
    fork = dict(op="fork", Hkv=4, D=256, Hv=16, reserve=22)
    comp = dict(op="compact", Hkv=4, D=256, sinks=4)
    return [
        # the smallest verify step of one sequence: latency
        dict(win, name="window-tiny", dtype="f16", Hq=8, Hkv=2, D=128, B=1, N=8, ctx=1024, ragged=False, window=256,
             sinks=4, trimmed=False),
        # plain decoding, one new token for each of 16 sequences
        dict(win, name="window-decode", B=16, N=1, ctx=32768, ragged=True, window=4096, sinks=4),
        # one sequence's verify step at budget 22 deep in a long context
        dict(win, name="window-verify-b22", B=1, N=22, ctx=131072, ragged=False, window=4096, sinks=4),
        # small groups, small odd window, sinks past one page, some sequences shorter than the window
        dict(win, name="window-odd", dtype="f16", Hq=15, Hkv=5, D=128, B=7, N=13, ctx=1500, ragged=True, window=777,
             sinks=70, trimmed=False),
        # a served batch of verify steps with a wide window: the largest
        dict(win, name="window-batch", B=32, N=22, ctx=16384, ragged=True, window=8192, sinks=64),
        # a toy vocabulary, one request of four beams: latency
        dict(beam, name="beam-tiny", B=1, K=4, Kout=4, V=4096),
        # eight requests of eight beams over a 27B-class vocabulary
        dict(beam, name="beam-b8-k8", B=8, K=8, Kout=8),
        # 16-bit logits, finished beams among the live ones, a grammar's mask over the vocabulary
        dict(beam, name="beam-b32-k8-bf16", dtype="bf16", B=32, K=8, Kout=8, done=True, masked=True),
        # one prompt becomes four beams
        dict(fork, name="fork-prompt", groups=1, K=1, Kout=4, ctx=1000, shared=0.0),
        # 24 requests of 8 beams each take their parents' pages and recurrent states
        dict(fork, name="fork-beams", groups=24, K=8, Kout=8, ctx=4096, shared=0.75),
        # one sequence's pages behind its window given back, the pool closed up
        dict(comp, name="compact-one", B=1, ctx=4000, window=1024, spare=64),
        # a served batch
        dict(comp, name="compact-batch", B=32, ctx=12000, window=4096, spare=512),
    ]


def _log(rng, lo, hi):
    return int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["window", "window", "beam", "fork", "compact"])
    if op == "window":
        Hkv, G = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 6, 8])
        D, N = rng.choice([128, 256]), _log(rng, 1, 64)
        window = _log(rng, 1, 8192)
        cap = 32 * 8192 * 4 * 256 // (min(window + 64, 16384) * Hkv * D)  # no more keys than the largest case
        B = _log(rng, 1, max(1, min(64, cap * 132 // max(132, N * G))))
        return dict(op=op, dtype=rng.choice(["bf16", "f16"]), Hq=Hkv * G, Hkv=Hkv, D=D, chain=rng.random() < 0.3,
                    trimmed=rng.random() < 0.5, B=B, N=N, ctx=_log(rng, 1, 16384), ragged=rng.random() < 0.7,
                    window=window, sinks=rng.choice([0, 1, 4, 64, rng.randint(0, 200)]))
    if op == "beam":
        K, Kout = _log(rng, 1, 32), _log(rng, 1, 32)
        V = _log(rng, 64, 151936)
        B = _log(rng, 1, max(1, min(32, 256 * 151936 // (K * V))))
        return dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]), B=B, K=K, Kout=Kout, V=V,
                    done=rng.random() < 0.5, masked=rng.random() < 0.5)
    if op == "fork":
        K, Kout = _log(rng, 1, 8), _log(rng, 1, 8)
        return dict(op=op, Hkv=rng.choice([1, 2, 4]), D=rng.choice([128, 256]), Hv=_log(rng, 1, 16),
                    reserve=_log(rng, 1, 64), groups=_log(rng, 1, 24), K=K, Kout=Kout, ctx=_log(rng, 1, 4096),
                    shared=rng.choice([0.0, 0.5, rng.random()]))
    return dict(op=op, Hkv=rng.choice([1, 2, 4]), D=rng.choice([128, 256]), sinks=rng.choice([0, 4, 64, 100]),
                B=_log(rng, 1, 32), ctx=_log(rng, 64, 12000), window=_log(rng, 1, 4096), spare=_log(rng, 8, 512))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _lengths(case, rng):
    B, ctx = case["B"], case["ctx"]
    if not case.get("ragged", True):
        return np.full(B, ctx)
    L = [ctx - i * (ctx // 2) // B for i in range(B)]  # the same lengths for every seed, in another order
    rng.shuffle(L)
    return np.array(L)


def _pools(pages, case, dtype, g):
    shape = (pages, case["Hkv"], PAGE, case["D"])
    return tuple(torch.randn(shape, generator=g, device="cuda", dtype=dtype) for _ in range(2))


def _prepare_window(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    dtype = DTYPES[case["dtype"]]
    L = _lengths(case, rng)
    per = -(-(L + N) // PAGE)
    maxp = int(per.max())
    pages = int(per.sum()) + 3
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table = np.full((B, maxp), -1)
    at = 0
    for b in range(B):
        table[b, :per[b]] = ids[at:at + per[b]]
        at += per[b]
        if case["trimmed"]:  # what lies behind the window has been given back
            table[b, -(-case["sinks"] // PAGE):max(0, int(L[b]) - case["window"] + 1) // PAGE] = -1
    parent = np.empty((B, N), np.int64)
    anc = np.zeros((B, N), np.uint64)
    for b in range(B):
        for i in range(N):
            p = i - 1 if case["chain"] or i == 0 else rng.randint(0, i - 1)
            parent[b, i] = p
            anc[b, i] = np.uint64(1 << i) | (anc[b, p] if p >= 0 else np.uint64(0))
    k_pool, v_pool = _pools(pages, case, dtype, g)
    n = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    return dict(q=n(B, N, Hq, D), k_pool=k_pool, v_pool=v_pool, page_table=_int(table), ctx_len=_int(L),
                k_tree=n(B, N, Hkv, D), v_tree=n(B, N, Hkv, D),
                anc_mask=torch.from_numpy(anc.view(np.int64)).cuda(), parent=parent, window=case["window"],
                sinks=case["sinks"])


def _prepare_beam(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    B, K, V, dtype = case["B"], case["K"], case["V"], DTYPES[case["dtype"]]
    logits = (3 * torch.randn(B, K, V, generator=g, device="cuda")).to(dtype)
    if case["masked"]:  # a grammar leaves some of the vocabulary
        logits.masked_fill_(torch.rand(B, 1, V, generator=g, device="cuda") < 0.9, float("-inf"))
    cum = -20 * torch.rand(B, K, generator=g, device="cuda") - 1
    finished = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    if case["done"]:
        finished = (torch.rand(B, K, generator=g, device="cuda") < 0.25).to(torch.int32)
    return dict(logits=logits, cum=cum, finished=finished, eos=rng.randrange(V), Kout=min(case["Kout"], K * V))


def _prepare_fork(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    G, K, Kout, reserve = case["groups"], case["K"], case["Kout"], case["reserve"]
    L = _lengths(dict(B=G, ctx=case["ctx"]), rng)
    per, full = -(-(L + reserve) // PAGE), L // PAGE
    both = (full * case["shared"]).astype(int)
    tail = -(-(L + reserve) // PAGE) - full
    used = int((both + K * (per - both)).sum())
    pages = used + int((Kout * (tail + 1)).sum()) + 5
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table, ref = np.full((G * K, int(per.max())), -1), np.zeros(pages, int)
    at = 0
    for j in range(G):
        pre = ids[at:at + both[j]]
        at += both[j]
        ref[pre] = K
        for k in range(K):
            mine = ids[at:at + per[j] - both[j]]
            at += len(mine)
            ref[mine] = 1
            table[j * K + k, :per[j]] = np.concatenate([pre, mine])
    src = np.array([j * K + rng.randrange(K) for j in range(G) for _ in range(Kout)])
    k_pool, v_pool = _pools(pages, case, torch.bfloat16, g)
    state = torch.randn(G * K, case["Hv"], 128, 128, generator=g, device="cuda")
    return dict(table=_int(table), ctx=_int(np.repeat(L, K)), src=_int(src), reserve=reserve, ref=_int(ref),
                k_pool=k_pool, v_pool=v_pool, state=state)


def _prepare_compact(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    B = case["B"]
    L = _lengths(case, rng)
    per = -(-L // PAGE)
    both = [int(per[b - 1].item() // 2) if b % 2 and per[b] >= per[b - 1] // 2 else 0 for b in range(B)]
    pages = int(per.sum()) + case["spare"]
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table, ref = np.full((B, int(per.max()) + 1), -1), np.zeros(pages, int)
    at = 0
    for b in range(B):  # odd rows share the first half of the row before them
        table[b, :both[b]] = table[b - 1, :both[b]]
        table[b, both[b]:per[b]] = ids[at:at + per[b] - both[b]]
        at += per[b] - both[b]
        ref[table[b, :per[b]]] += 1
    k_pool, v_pool = _pools(pages, case, torch.bfloat16, g)
    return dict(table=_int(table), ctx=_int(L), ref=_int(ref), k_pool=k_pool, v_pool=v_pool, window=case["window"],
                sinks=case["sinks"])


def prepare(case, seed):
    s = dict(globals()["_prepare_" + case["op"]](case, seed), op=case["op"])
    if own:
        _buffers(s)
    return s


# ------------------------------------------------------------------ the library's calls

def _buffers(s):
    """The outputs and workspaces that a serving program keeps."""
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    e = lambda *shape, t=torch.int32: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if s["op"] == "window":
        B, N, Hq, D = s["q"].shape
        s["out"], s["lse"] = e(B, N, Hq, D, t=s["q"].dtype), e(B, N, Hq, t=torch.float32)
        s["ws"] = e(LT.lucetree_verify_attn_workspace(B, N, Hq, s["k_tree"].shape[2], D), t=torch.uint8)
    elif s["op"] == "beam":
        B, K, V = s["logits"].shape
        s["score"] = e(B, s["Kout"], t=torch.float32)
        s["token"], s["row"], s["done"] = (e(B, s["Kout"]) for _ in range(3))
        s["ws"] = e(LT.lucetree_beam_select_workspace(B, K, s["Kout"], V), t=torch.uint8)
    elif s["op"] == "fork":
        R, P, n = s["src"].numel(), s["table"].shape[1], s["ref"].numel()
        s["table_out"], s["ctx_out"], s["ref_out"] = e(R, P), e(R), e(n)
        s["copy_src"], s["copy_dst"] = e(R), e(R)
        s["state_out"] = e(R, *s["state"].shape[1:], t=torch.float32)
        s["ws"] = e(LT.lucetree_reorder_pages_workspace(s["table"].shape[0], R, n), t=torch.uint8)
    else:
        n = s["ref"].numel()
        s["table_out"], s["ref_out"], s["live"] = e(*s["table"].shape), e(n), e(1)
        s["copy_src"], s["copy_dst"], s["copy_n"] = e(n // 2), e(n // 2), e(1)
        s["ws"] = e(LT.lucetree_compact_pages_workspace(n), t=torch.uint8)


def _own(s):
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    st = s["status"]
    if s["op"] == "window":
        LT.lucetree_verify_attn_win(s["q"], s["k_pool"], s["v_pool"], s["page_table"], s["ctx_len"], s["k_tree"],
                                    s["v_tree"], s["anc_mask"], s["window"], s["sinks"], s["out"], st, s["ws"],
                                    lse=s["lse"])
        return s["out"], s["lse"]
    if s["op"] == "beam":
        LT.lucetree_beam_select(s["logits"], s["cum"], s["finished"], s["eos"], s["score"], s["token"], s["row"],
                                s["done"], s["ws"])
        return s["score"], s["token"], s["row"], s["done"]
    if s["op"] == "fork":
        LT.lucetree_reorder_pages(s["table"], s["ctx"], s["src"], s["reserve"], s["ref"], s["table_out"], s["ctx_out"],
                                  s["ref_out"], s["copy_src"], s["copy_dst"], st, s["ws"])
        LT.lucetree_copy_pages(s["copy_src"], s["copy_dst"], s["k_pool"], s["v_pool"], st)
        LT.lucetree_reorder_states(s["state"], s["src"], s["state_out"], st)
        return (s["table_out"], s["ctx_out"], s["ref_out"], s["copy_src"], s["copy_dst"], s["k_pool"], s["v_pool"],
                s["state_out"])
    LT.lucetree_trim_pages(s["table"], s["ctx"], s["window"], s["sinks"], s["ref"], s["table_out"], s["ref_out"], st)
    LT.lucetree_compact_pages(s["table_out"], s["ref_out"], s["table_out"], s["ref_out"], s["copy_src"], s["copy_dst"],
                              s["copy_n"], s["live"], st, s["ws"])
    LT.lucetree_copy_pages(s["copy_src"], s["copy_dst"], s["k_pool"], s["v_pool"], st, count=s["copy_n"])
    return s["table_out"], s["ref_out"], s["copy_src"], s["copy_dst"], s["live"], s["k_pool"], s["v_pool"]


# ------------------------------------------------------------------ the plain forms

def _plain_window(s):
    q, L, W, S = s["q"].float(), s["ctx_len"].long(), s["window"], s["sinks"]
    B, N, Hq, D = q.shape
    Hkv = s["k_tree"].shape[2]
    G, maxp = Hq // Hkv, s["page_table"].shape[1]
    # the committed positions that any node can see: the sinks, then the window of a node at depth 0
    first = (L - W + 1).clamp(min=0)
    n_sink, n_win = min(S, maxp * PAGE), min(W, maxp * PAGE)
    j = torch.arange(n_sink + n_win, device=q.device)
    is_sink = j < n_sink
    pos = torch.where(is_sink, j, first[:, None] + j - n_sink)                                       # [B][M]
    there = (pos < L[:, None]) & (is_sink | (pos >= n_sink))
    page = torch.gather(s["page_table"].long(), 1, (pos // PAGE).clamp(max=maxp - 1))
    there &= page >= 0
    page = page.clamp(min=0)
    k = s["k_pool"][page, :, pos % PAGE].float()                                                     # [B][M][Hkv][D]
    v = s["v_pool"][page, :, pos % PAGE].float()
    bit = torch.arange(N, device=q.device)
    sees = ((s["anc_mask"][:, :, None] >> bit) & 1).bool()                                           # [B][N][N]
    at = L[:, None] + sees.sum(-1) - 1                                                               # node positions
    ok = there[:, None] & ((pos[:, None] < S) | (at[:, :, None] - pos[:, None] < W))                 # [B][N][M]
    ok_tree = sees & ((at[:, None, :] < S) | (at[:, :, None] - at[:, None, :] < W))
    q = q.view(B, N, Hkv, G, D) * D ** -0.5
    scores = torch.cat([torch.einsum("bngxd,bmgd->bgxnm", q, k),
                        torch.einsum("bngxd,bmgd->bgxnm", q, s["k_tree"].float())], -1)
    ok = torch.cat([ok, ok_tree], -1)[:, None, None]
    scores = torch.where(ok, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1)                                                                                # [B][Hkv][G][N]
    M = pos.shape[1]
    out = torch.einsum("bgxnm,bmgd->bngxd", p[..., :M], torch.where(there[:, :, None, None], v, 0.0)) + \
        torch.einsum("bgxnm,bmgd->bngxd", p[..., M:], s["v_tree"].float())
    out = out / total.permute(0, 3, 1, 2)[..., None]
    lse = (top[..., 0] + torch.log(total)).permute(0, 3, 1, 2)
    return out.reshape(B, N, Hq, D).to(s["q"].dtype), lse.reshape(B, N, Hq)


def _plain_beam(s):
    # 64 bits: neighbouring candidates of different beams differ by less than fp32 keeps beside a long sum
    x, cum = s["logits"].double(), s["cum"].double()
    B, K, V = x.shape
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    score = torch.where(torch.isinf(x), float("-inf"), x - lse) + cum[..., None]
    fin = s["finished"].bool()[..., None]
    ends = torch.arange(V, device=x.device) == s["eos"]
    score = torch.where(fin, torch.where(ends, cum[..., None], float("-inf")), score)
    score, order = torch.sort(score.view(B, K * V), dim=-1, descending=True, stable=True)
    score, order = score[:, :s["Kout"]], order[:, :s["Kout"]]
    token, beam = order % V, order // V
    row = beam + K * torch.arange(B, device=x.device)[:, None]
    done = s["finished"].view(-1)[row].bool() | (token == s["eos"])
    return score.float(), token.int(), row.int(), done.int()


def _plain_copy(src, dst, k_pool, v_pool):
    at = (src >= 0) & (dst >= 0)
    src, dst = src[at].long(), dst[at].long()
    k_pool[dst], v_pool[dst] = k_pool[src], v_pool[src]


def _plain_fork(s):
    table, src, ref, reserve = s["table"].long(), s["src"].long(), s["ref"].long(), s["reserve"]
    (R, P), rows, pages = table.shape, s["src"].numel(), s["ref"].numel()
    L = s["ctx"].long()
    col = torch.arange(P, device=src.device)
    full, end = (L // PAGE)[:, None], ((L + reserve + PAGE - 1) // PAGE)[:, None]                     # of each old row
    r = torch.arange(rows, device=src.device)
    children = torch.zeros(R, dtype=torch.long, device=src.device).index_add_(0, src, torch.ones_like(src))
    first = torch.full((R,), rows, device=src.device).scatter_reduce_(0, src, r, "amin")
    mapped, page = table >= 0, table.clamp(min=0)
    old_tail = (col >= full) & (col < end)
    kept = old_tail & mapped & (ref[page] == 1) & (children > 0)[:, None]
    delta = torch.where(col < full, (children - 1)[:, None], torch.where(kept, 0, -1)) * mapped
    new_ref = ref.index_add(0, page.view(-1), delta.view(-1))
    # new rows
    keep = kept[src] & (first[src] == r)[:, None]
    fresh = old_tail[src] & ~keep
    rank = (torch.cumsum(fresh.view(-1).long(), 0) - 1).view(rows, P)
    free = torch.sort((ref != 0).int(), stable=True).indices
    new = torch.where(rank < (ref == 0).sum(), free[rank.clamp(0, pages - 1)], -1)
    out = torch.where((col < full[src]) | keep, table[src], torch.where(fresh, new, -1))
    new_ref = new_ref.index_add(0, torch.where(fresh, new, 0).clamp(min=0).view(-1), (fresh & (new >= 0)).view(-1).long())
    at = full[src].clamp(max=P - 1)
    take = lambda t: torch.gather(t, 1, at)[:, 0]  # noqa: E731
    copies = (L[src] % PAGE > 0) & take(fresh) & (take(table[src]) >= 0) & (take(out) >= 0)
    copy_src = torch.where(copies, take(table[src]), -1).int()
    copy_dst = torch.where(copies, take(out), -1).int()
    _plain_copy(copy_src, copy_dst, s["k_pool"], s["v_pool"])
    return (out.int(), s["ctx"][src], new_ref.int(), copy_src, copy_dst, s["k_pool"], s["v_pool"], s["state"][src])


def _plain_compact(s):
    table, ref, L = s["table"].long(), s["ref"].long(), s["ctx"].long()
    pages = ref.numel()
    col = torch.arange(table.shape[1], device=ref.device)
    behind = (col >= -(-s["sinks"] // PAGE)) & ((col + 1) * PAGE <= (L - s["window"] + 1)[:, None])
    gone = behind & (table >= 0)
    ref = ref.index_add(0, table.clamp(min=0).view(-1), -gone.view(-1).long())
    table = torch.where(behind, -1, table)
    ids = torch.arange(pages, device=ref.device)
    used = ref > 0
    live = used.sum()
    half = ids[:pages // 2]
    mover, hole = used & (ids >= live), ~used & (ids < live)
    frm, to = (torch.sort((~m).int(), stable=True).indices[:pages // 2] for m in (mover, hole))
    moves = half < mover.sum()
    name = ids.scatter(0, frm, torch.where(moves, to, frm))
    table = torch.where(table >= 0, name[table.clamp(min=0)], -1)
    rank = (torch.cumsum(hole.long(), 0) - 1).clamp(0, pages // 2 - 1)
    new_ref = torch.where(hole, ref[frm[rank]], torch.where(ids < live, ref, 0))
    copy_src, copy_dst = torch.where(moves, frm, -1).int(), torch.where(moves, to, -1).int()
    _plain_copy(copy_src, copy_dst, s["k_pool"], s["v_pool"])
    return table.int(), new_ref.int(), copy_src, copy_dst, live.int().view(1), s["k_pool"], s["v_pool"]


def run(state):
    if own:
        return _own(state)
    return globals()["_plain_" + state["op"]](state)


# ------------------------------------------------------------------ what cannot be done without

def work(case):
    """Means of the drawn lengths where they are ragged."""
    mean = 0.75 if case.get("ragged", True) else 1.0
    if case["op"] == "window":
        B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
        L = mean * case["ctx"]
        keys = L if L <= case["window"] + case["sinks"] else case["window"] + case["sinks"]
        rows = B * N * Hq
        return {"bytes": B * keys * Hkv * D * 4 + rows * D * 4 + B * N * Hkv * D * 4 + rows * 4 + 8 * B * N,
                "flops": 4.0 * rows * D * (keys + 1)}
    if case["op"] == "beam":
        n = case["B"] * case["K"] * case["V"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["B"] * (8 * case["K"] + 16 * case["Kout"]),
                "flops": 4.0 * n}
    page = 2 * 2 * PAGE * case["Hkv"] * case["D"]
    if case["op"] == "fork":
        rows, old = case["groups"] * case["Kout"], case["groups"] * case["K"]
        cols = (mean * case["ctx"] + case["reserve"]) / PAGE
        # of the children of a group's K beams, all but one for each beam that has any need a copied page
        copies = case["groups"] * (case["Kout"] - case["K"] * (1 - (1 - 1 / case["K"]) ** case["Kout"]))
        states = (rows + old * (1 - (1 - 1 / case["K"]) ** case["Kout"])) * case["Hv"] * 128 * 128 * 4
        return {"bytes": 2 * copies * page + states + 4 * cols * (rows + old) + 16 * rows, "flops": 0}
    cols = mean * case["ctx"] / PAGE
    pages = case["B"] * cols * 0.75 + case["spare"]
    left = case["B"] * min(cols, (case["window"] + min(case["sinks"], 2 * PAGE)) / PAGE + 1)
    return {"bytes": 2 * page * left * max(0.0, 1 - left / pages) + 8 * case["B"] * cols + 8 * pages, "flops": 0}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_window(case, seed):
    s = _prepare_window(case, seed)
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    out = torch.empty(B, N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, N, Hq, dtype=torch.float64, device="cuda")
    for b in range(B):
        L = int(s["ctx_len"][b])
        paths = []
        for i in range(N):
            path, c = [], i
            while c >= 0:
                path.append(c)
                c = int(s["parent"][b, c])
            paths.append(path)
        keys = torch.arange(L, device="cuda")
        at = torch.tensor([L + len(p) - 1 for p in paths], device="cuda")
        see = (keys < case["sinks"]) | (keys > (at - case["window"])[:, None])                       # [N][L]
        sel = torch.nonzero(see.any(0))[:, 0]
        pages = s["page_table"][b][sel // PAGE].long()
        mask = np.zeros((N, N), bool)
        for i, path in enumerate(paths):
            for j in path:
                mask[i, j] = int(at[i] - at[j]) < case["window"] or int(at[j]) < case["sinks"]
        mask = torch.cat([see[:, sel], torch.from_numpy(mask).cuda()], 1)
        for g in range(Hkv):
            k = torch.cat([s["k_pool"][pages, g, sel % PAGE], s["k_tree"][b, :, g]]).double()
            v = torch.cat([s["v_pool"][pages, g, sel % PAGE], s["v_tree"][b, :, g]]).double()
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                t = (s["q"][b, :, h].double() @ k.T / D ** 0.5).masked_fill(~mask, float("-inf"))
                lse[b, :, h] = torch.logsumexp(t, -1)
                out[b, :, h] = torch.exp(t - lse[b, :, h, None]) @ v
    return out, lse


def _exact_beam(case, seed):
    s = _prepare_beam(case, seed)
    x = s["logits"].double().cpu().numpy()
    cum, fin = s["cum"].double().cpu().numpy(), s["finished"].cpu().numpy()
    B, K, V = x.shape
    Kout, got = s["Kout"], ([], [], [], [])
    for b in range(B):
        cands = []
        for k in range(K):
            if fin[b, k]:
                sc = np.full(V, -np.inf)
                sc[s["eos"]] = cum[b, k]
            else:
                with np.errstate(divide="ignore", invalid="ignore"):
                    m = x[b, k].max()
                    sc = x[b, k] - (m + np.log(np.exp(x[b, k] - m).sum())) + cum[b, k]
                sc[np.isnan(sc)] = -np.inf
            best = np.argsort(-sc, kind="stable")[:Kout]
            cands += [(-sc[t], k * V + int(t)) for t in best]
        cands = sorted(cands)[:Kout]
        got[0].append([-c for c, _ in cands])
        got[1].append([i % V for _, i in cands])
        got[2].append([b * K + i // V for _, i in cands])
        got[3].append([int(fin[b, i // V] != 0 or i % V == s["eos"]) for _, i in cands])
    return (np.array(got[0]),) + tuple(np.array(a, np.int32) for a in got[1:])


def _exact_fork(case, seed):
    s = _prepare_fork(case, seed)
    table, ctx, src = (s[k].cpu().numpy() for k in ("table", "ctx", "src"))
    ref = s["ref"].cpu().numpy().copy()
    free = [int(p) for p in np.nonzero(ref == 0)[0]]
    held, out, pairs, taken = ref.copy(), np.full((len(src), table.shape[1]), -1), [], set()
    for b in range(len(ctx)):  # the old rows let go
        for p in table[b]:
            ref[p] -= p >= 0
    for r, b in enumerate(src):
        L = int(ctx[b])
        pair = (-1, -1)
        for c in range(-(-(L + s["reserve"]) // PAGE)):
            p = int(table[b, c])
            if c >= L // PAGE and not (p >= 0 and held[p] == 1 and b not in taken):
                new = free.pop(0)
                if c == L // PAGE and L % PAGE and p >= 0:
                    pair = (p, new)
                p = new
            out[r, c] = p
            ref[p] += p >= 0
        taken.add(b)
        pairs.append(pair)
    frm, to = np.array(pairs, np.int32).T
    at = torch.from_numpy(np.nonzero(frm >= 0)[0])
    pools = []
    for name in ("k_pool", "v_pool"):
        pool = s[name]
        for i in at.tolist():
            pool[int(to[i])].copy_(pool[int(frm[i])])
        pools.append(pool)
    state = torch.stack([s["state"][int(b)] for b in src])
    return out.astype(np.int32), ctx[src], ref, frm, to, pools[0], pools[1], state


def _exact_compact(case, seed):
    s = _prepare_compact(case, seed)
    table, ctx, ref = s["table"].cpu().numpy().copy(), s["ctx"].cpu().numpy(), s["ref"].cpu().numpy().copy()
    for b in range(table.shape[0]):
        for c in range(table.shape[1]):
            if c * PAGE >= s["sinks"] and (c + 1) * PAGE - 1 <= int(ctx[b]) - s["window"]:
                if table[b, c] >= 0:
                    ref[table[b, c]] -= 1
                table[b, c] = -1
    live = int((ref > 0).sum())
    holes = [p for p in range(live) if ref[p] <= 0]
    movers = [p for p in range(live, len(ref)) if ref[p] > 0]
    name = {p: h for p, h in zip(movers, holes)}
    new_table = np.array([[name.get(int(p), int(p)) for p in row] for row in table], np.int32)
    frm, to = np.full(len(ref) // 2, -1, np.int32), np.full(len(ref) // 2, -1, np.int32)
    new_ref = ref.copy()
    for i, (p, h) in enumerate(name.items()):
        frm[i], to[i] = p, h
        new_ref[h], new_ref[p] = ref[p], 0
        for pool in ("k_pool", "v_pool"):
            s[pool][h].copy_(s[pool][p])
    return new_table, new_ref, frm, to, np.array([live], np.int32), s["k_pool"], s["v_pool"]


def exact(case, seed):
    return globals()["_exact_" + case["op"]](case, seed)
