"""Cases and plain forms of the operators around a shared, growing cache: rotary
positions of tree nodes, appending keys and values to the paged cache, and
tree-verify attention of a batch that shares prefixes.

``own`` chooses what ``run`` computes: False, the plain form in elementary
torch operations; True, the library's calls on the same inputs.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    rope = dict(op="rope", dtype="bf16", Hq=24, Hkv=4, D=256, layout="half", scaling="none", factor=1.0)
    app = dict(op="append", dtype="bf16", Hq=24, Hkv=4, D=256, rot=256, layout="half", scaling="none", factor=1.0,
               store="same")
    att = dict(op="shared", dtype="bf16", Hq=24, Hkv=4, D=256)
    return [
        # the draft tree of one sequence: latency
        dict(rope, name="rope-one", dtype="f16", Hq=8, Hkv=2, D=128, rot=128, B=1, N=8, ctx=1024),
        # a served batch of verify steps deep in a stretched context, a quarter of the head rotated
        dict(rope, name="rope-batch", rot=64, scaling="yarn", factor=4.0, B=32, N=22, ctx=131072),
        # one decoded token for each of 16 sequences
        dict(app, name="append-decode", B=16, new=1, ragged=False, ctx=32768),
        # adjacent pairs, small groups, odd prompts
        dict(app, name="append-odd", dtype="f16", Hq=15, Hkv=5, D=128, rot=96, layout="pairs", scaling="bands",
             factor=8.0, B=7, new=333, ragged=True, ctx=1500),
        # prompts of a served batch: the largest
        dict(app, name="append-prompts", B=8, new=4096, ragged=True, ctx=0),
        # a chunk of each prompt into a quantised cache
        dict(app, name="append-quantised", scaling="ntk", factor=2.0, B=16, new=512, ragged=True, ctx=2048, store="kq-v8"),
        # four continuations of a short prompt: latency
        dict(att, name="shared-four", dtype="f16", Hq=8, Hkv=2, D=128, B=4, N=1, groups=1, prefix=512, private=64),
        # 32 sampled answers to one long prompt, one token each
        dict(att, name="shared-decode", B=32, N=1, groups=1, prefix=32768, private=1024),
        # beams: 24 requests of some eight beams
        dict(att, name="shared-beams", B=192, N=1, groups=24, prefix=4096, private=256),
        # small groups of verify steps, some sequences alone
        dict(att, name="shared-odd", dtype="f16", Hq=15, Hkv=5, D=128, B=21, N=13, groups=9, prefix=3000, private=777),
        # verify steps of 16 sequences under one long system prompt: the largest
        dict(att, name="shared-verify", B=16, N=22, groups=1, prefix=16384, private=2048),
    ]


def _log(rng, lo, hi):
    return int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi + 0.49))))))


def _draw_rope(rng, D):
    layout = rng.choice(["half", "pairs"])
    rot = rng.choice([D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
    scaling = rng.choice(["none", "linear", "ntk", "bands", "yarn"]) if rot > 2 else "none"
    return dict(layout=layout, rot=rot, scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "shared", "shared", "shared"])
    Hkv, G = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 6, 8])
    D, dtype = rng.choice([128, 256]), rng.choice(["bf16", "f16"])
    heads = dict(Hq=Hkv * G, Hkv=Hkv, D=D)
    if op == "rope":
        return dict(heads, op=op, dtype=dtype, B=_log(rng, 1, 32), N=_log(rng, 1, 22), ctx=_log(rng, 1, 131072),
                    **_draw_rope(rng, D))
    if op == "append":
        store = rng.choice(["same", "same", "v8", "v4", "kq", "kq-v8", "kq-v4"])
        if store != "same":
            heads["D"] = D = 256
            dtype = "bf16" if store[0] == "k" else dtype
        most = 8 * 4096 * 32 * 256 // ((Hkv * G + 2 * Hkv) * D)  # the largest case's elements
        new = _log(rng, 1, min(4096, most))
        return dict(heads, op=op, dtype=dtype, B=_log(rng, 1, max(1, min(64, most // new))), new=new,
                    ragged=rng.random() < 0.7, ctx=rng.choice([0, _log(rng, 1, 4096)]), store=store, **_draw_rope(rng, D))
    B = _log(rng, 1, 192)
    groups = min(B, _log(rng, 1, 24))
    N = _log(rng, 1, 64)
    # no more products than the largest case, and no more keys than the plain form can hold for all rows
    cap = min(16 * 22 * 24 * 18432 * 256 // (B * N * Hkv * G * D), 32 * 34000 * 4 * 256 // (B * Hkv * D))
    prefix = _log(rng, 1, max(1, min(32768, cap * 7 // 8)))
    return dict(heads, op=op, dtype=dtype, B=B, N=N, groups=groups, prefix=prefix,
                private=_log(rng, 1, max(1, min(2048, cap - prefix))))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _spread(n, top, low, rng):
    """n whole numbers from top down to low, in an order of their own for each seed."""
    x = [top - i * (top - low) // max(1, n) for i in range(n)]
    rng.shuffle(x)
    return np.array(x)


def _projected(rows, case, g):
    """The queries, keys and values of `rows` tokens as a projection leaves them: one row after the other."""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    x = torch.randn(*rows, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    return tuple(t.unflatten(-1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], -1))


def _masks(B, N, rng):
    anc = np.zeros((B, N), np.uint64)
    for b in range(B):
        for i in range(N):
            p = rng.randint(-1, i - 1) if i else -1
            anc[b, i] = np.uint64(1 << i) | (anc[b, p] if p >= 0 else np.uint64(0))
    return torch.from_numpy(anc.view(np.int64)).cuda()


def _prepare_rope(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    B, N = case["B"], case["N"]
    q, k, v = _projected((B, N), case, g)
    return dict(q=q, k=k, v=v, ctx_len=_int(_spread(B, case["ctx"], case["ctx"] // 2, rng)), anc_mask=_masks(B, N, rng))


def _pools(pages, case, g):
    """Pools that have been in use: what stands in them stays where nothing is appended."""
    Hkv, D, store, t = case["Hkv"], case["D"], case["store"], DTYPES[case["dtype"]]
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    s = {}
    for name, fmt in (("k", "e4m3" if "kq" in store else "same"),
                      ("v", "int8" if "v8" in store else "int4" if "v4" in store else "same")):
        if fmt == "same":
            s[name + "_pool"] = torch.randn(pages, Hkv, PAGE, D, generator=g, device="cuda").to(t)
        else:
            s[name + "_pool"] = byte(1, 120, pages, Hkv, PAGE, D // 2 if fmt == "int4" else D)
            s[name + "_exp"] = byte(115, 125, pages, Hkv, PAGE)
    return s


def _prepare_append(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    B, new, ctx = case["B"], case["new"], case["ctx"]
    n = _spread(B, new, new // 2, rng) if case["ragged"] else np.full(B, new)
    L = _spread(B, ctx, ctx // 2, rng)
    start = np.concatenate([[0], np.cumsum(n)])
    first, per = L // PAGE, -(-(L + n) // PAGE)
    # only the pages that the new tokens reach: what lies before them stays out of the case
    pages = B * (-(-new // PAGE) + 1) + 3
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table = np.full((B, int(-(-(ctx + new) // PAGE))), -1)
    at = 0
    for b in range(B):
        table[b, first[b]:per[b]] = ids[at:at + per[b] - first[b]]
        at += per[b] - first[b]
    q, k, v = _projected((int(start[-1]),), case, g)
    return dict(q=q, k=k, v=v, start=_int(start), page_table=_int(table), ctx_len=_int(L), store=case["store"],
                **_pools(pages, case, g))


def _grouped(case, seed, rng):
    """Lengths, group borders and page tables of sequences of which each group has one prompt in common."""
    B, groups, N, private = case["B"], case["groups"], case["N"], case["private"]
    size = np.array([B // groups + (1 if g < B % groups else 0) for g in range(groups)])
    for g in range(1, groups, 2):  # groups of unlike sizes
        move = int(size[g]) // 2
        size[g] -= move
        size[g - 1] += move
    size = size[size > 0]
    rng.shuffle(size)
    start = np.concatenate([[0], np.cumsum(size)])
    prompt = np.repeat(_spread(len(size), case["prefix"], case["prefix"] // 2, rng), size)
    L = prompt + _spread(B, private, 0, rng)
    both, per = prompt // PAGE, -(-(L + N) // PAGE)
    table = np.full((B, int(-(-(case["prefix"] + private + N) // PAGE))), -1)
    firsts = np.repeat(start[:-1], size)
    pages = sum(-(-int(l + N) // PAGE) for l in L) + 3 if len(size) == B else \
        int(both[start[:-1]].sum() + (per - both).sum()) + 3
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    at = 0
    for b in range(B):
        lo = 0
        if firsts[b] != b:
            lo = int(both[b])
            table[b, :lo] = table[firsts[b], :lo]
        table[b, lo:per[b]] = ids[at:at + per[b] - lo]
        at += per[b] - lo
    return L, start, table, pages


def _prepare_shared(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    L, start, table, pages = _grouped(case, seed, rng)
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    t = DTYPES[case["dtype"]]
    n = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=t)  # noqa: E731
    return dict(q=n(B, N, Hq, D), k_pool=n(pages, Hkv, PAGE, D), v_pool=n(pages, Hkv, PAGE, D), page_table=_int(table),
                ctx_len=_int(L), group_start=_int(start), k_tree=n(B, N, Hkv, D), v_tree=n(B, N, Hkv, D),
                anc_mask=_masks(B, N, rng))


def prepare(case, seed):
    s = dict(globals()["_prepare_" + case["op"]](case, seed), op=case["op"])
    if "rot" in case:
        s["rope"] = {k: case[k] for k in ("rot", "layout", "scaling", "factor")}
    if own:
        _keep(s)
    return s


# ------------------------------------------------------------------ the library's calls

BASE, ORIG, LOW, HIGH, FAST, SLOW = 10000.0, 4096, 1.0, 4.0, 32.0, 1.0  # of the scaled forms


def _keep(s):
    """What a serving program keeps: the rotation's steps, outputs, and workspaces."""
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    e = lambda *shape, t=torch.int32: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if "rope" in s:
        r = s["rope"]
        kind = getattr(LT, "LUCETREE_ROPE_" + r["scaling"].upper())
        low, high = (SLOW, FAST) if r["scaling"] == "yarn" else (LOW, HIGH)
        steps, s["magnitude"] = LT.lucetree_rope_steps(r["rot"], BASE, scaling=kind, factor=r["factor"], orig_ctx=ORIG,
                                                       low=low, high=high)
        s["steps"], s["layout"] = steps.cuda(), getattr(LT, "LUCETREE_ROPE_" + r["layout"].upper())
    if s["op"] == "rope":
        s["q_out"], s["k_out"], s["v_out"] = (e(*s[n].shape, t=s[n].dtype) for n in "qkv")
    elif s["op"] == "append":
        s["q_out"], s["ctx_out"] = e(*s["q"].shape, t=s["q"].dtype), e(*s["ctx_len"].shape)
    else:
        (B, N, Hq, D), Hkv, groups = s["q"].shape, s["k_tree"].shape[2], s["group_start"].numel() - 1
        s["heads"] = N, Hq, Hkv, D
        s["shared"], s["plan"] = e(groups), e(LT.lucetree_shared_plan_bytes(B, N, Hq, Hkv, D, groups), t=torch.uint8)
        s["out"], s["lse"] = e(*s["q"].shape, t=s["q"].dtype), e(B, N, Hq, t=torch.float32)
        s["ws"] = e(LT.lucetree_verify_attn_shared_workspace(B, N, Hq, Hkv, D, groups), t=torch.uint8)


def _own(s):
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    if s["op"] == "rope":
        LT.lucetree_rope(s["q"], s["k"], s["steps"], s["layout"], s["q_out"], s["k_out"], s["status"],
                         ctx_len=s["ctx_len"], anc_mask=s["anc_mask"], v=s["v"], v_out=s["v_out"],
                         magnitude=s["magnitude"])
        return s["q_out"], s["k_out"], s["v_out"]
    if s["op"] == "append":
        v_format = LT.LUCETREE_V_INT8 if "v8" in s["store"] else LT.LUCETREE_V_INT4 if "v4" in s["store"] else \
            LT.LUCETREE_V_SAME
        LT.lucetree_append_kv(s["k"], s["v"], s["start"], s["page_table"], s["ctx_len"], s["ctx_out"], s["k_pool"],
                              s["v_pool"], s["status"], q=s["q"], q_out=s["q_out"], steps=s["steps"],
                              layout=s["layout"], magnitude=s["magnitude"], k_exp=s.get("k_exp"), v_format=v_format,
                              v_exp=s.get("v_exp"))
        return s["q_out"], *_values(s), s["ctx_out"]
    LT.lucetree_shared_plan(s["page_table"], s["ctx_len"], s["group_start"], *s["heads"], s["k_pool"].shape[0],
                            s["shared"], s["plan"], s["status"])
    LT.lucetree_verify_attn_shared(s["q"], s["k_pool"], s["v_pool"], s["page_table"], s["ctx_len"], s["k_tree"],
                                   s["v_tree"], s["anc_mask"], s["group_start"].numel() - 1, s["plan"], s["out"],
                                   s["status"], s["ws"], lse=s["lse"])
    return s["out"], s["lse"]


# ------------------------------------------------------------------ the plain forms

def _values(s):
    """The pools as values: codes times their row's power of two, which bf16 holds exactly."""
    out = []
    for name in ("k", "v"):
        x = s[name + "_pool"]
        if name + "_exp" in s:
            if name == "k":
                x = x.view(torch.float8_e4m3fn).to(torch.bfloat16)
            elif "v8" in s["store"]:
                x = x.view(torch.int8).to(torch.bfloat16)
            else:
                x = x.view(torch.int8)
                x = torch.stack([(x << 4) >> 4, x >> 4], -1).flatten(-2).to(torch.bfloat16)
            e = s[name + "_exp"]
            x = x * torch.where(e > 0, torch.exp2(e.float() - 127), 0.0).to(torch.bfloat16)[..., None]
        out.append(x)
    return out


def _plain_frequencies(r):
    """(angle per position of each pair, magnitude); in 64 bits: far positions multiply what is lost here."""
    rot, factor = r["rot"], r["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = BASE ** (-2 * i / rot)
    if r["scaling"] == "linear":
        f = f / factor
    elif r["scaling"] == "ntk":
        f = (BASE * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
    elif r["scaling"] == "bands":
        turns = ORIG * f / (2 * math.pi)
        t = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = (1 - t) * f / factor + t * f
    elif r["scaling"] == "yarn":
        at = lambda n: rot * math.log(ORIG / (2 * math.pi * n)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(math.floor(at(FAST)), 0), min(math.ceil(at(SLOW)), rot - 1)
        ramp = ((i - lo) / (hi - lo if hi > lo else 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    return f, 1.0


def _plain_rotate(x, pos, r):
    """x [..., H, D] at positions pos [...]."""
    f, m = _plain_frequencies(r)
    t = pos.double()[..., None, None] * f
    cos, sin = (torch.cos(t) * m).float(), (torch.sin(t) * m).float()
    rot, h = r["rot"], r["rot"] // 2
    y, x = x.float(), x.float()
    if r["layout"] == "half":
        a, b = x[..., :h], x[..., h:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_rope(s):
    bits = torch.arange(s["anc_mask"].shape[1], device="cuda")
    depth = ((s["anc_mask"][..., None] >> bits) & 1).sum(-1) - 1
    pos = s["ctx_len"].long()[:, None] + depth
    return _plain_rotate(s["q"], pos, s["rope"]).to(s["q"].dtype), _plain_rotate(s["k"], pos, s["rope"]).to(s["k"].dtype), \
        s["v"].contiguous()


def _plain_scale(x, most):
    """The largest p with max|x| 2^p <= most (a power of two's multiple), of each row."""
    m = x.abs().amax(-1)
    p = torch.floor(torch.log2(most / torch.where(m > 0, m, 1.0)))
    p = torch.where(m * torch.exp2(p + 1) <= most, p + 1, p)  # (the logarithm is rounded)
    p = torch.where(m * torch.exp2(p) > most, p - 1, p)
    fine = (m > 0) & (p <= 126) & (p >= -127)
    return torch.where(fine, p, 0.0), fine


def _plain_append(s):
    start, L = s["start"].long(), s["ctx_len"].long()
    n = start[1:] - start[:-1]
    T, B = s["k"].shape[0], L.numel()
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), n, output_size=T)
    pos = L[seq] + torch.arange(T, device="cuda") - start[seq]
    page, slot = s["page_table"].long()[seq, pos // PAGE], pos % PAGE
    q = _plain_rotate(s["q"], pos, s["rope"]).to(s["q"].dtype)
    k, v = _plain_rotate(s["k"], pos, s["rope"]), s["v"]
    if "k_exp" in s:
        p, fine = _plain_scale(k, 448.0)
        code = (k * torch.exp2(p)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k_pool"][page, :, slot] = torch.where(fine[..., None], code, 0).to(torch.uint8)
        s["k_exp"][page, :, slot] = torch.where(fine, 127 - p, 0.0).to(torch.uint8)
    else:
        s["k_pool"][page, :, slot] = k.to(s["k"].dtype)
    if "v_exp" in s:
        p, fine = _plain_scale(v.float(), 127.0 if "v8" in s["store"] else 7.0)
        code = torch.round(v.float() * torch.exp2(p)[..., None]).to(torch.int8)
        code = torch.where(fine[..., None], code, 0)
        if "v4" in s["store"]:
            code = (code[..., 0::2] & 15) | (code[..., 1::2] << 4)
        s["v_pool"][page, :, slot] = code.view(torch.uint8)
        s["v_exp"][page, :, slot] = torch.where(fine, 127 - p, 0.0).to(torch.uint8)
    else:
        s["v_pool"][page, :, slot] = v
    return q, *_values(s), (L + n).int()


def _plain_shared(s):
    q, L = s["q"].float(), s["ctx_len"].long()
    B, N, Hq, D = q.shape
    Hkv = s["k_tree"].shape[2]
    maxp = s["page_table"].shape[1]
    pos = torch.arange(maxp * PAGE, device=q.device)
    there = pos < L[:, None]
    page = torch.where(there, s["page_table"].long().repeat_interleave(PAGE, 1), 0).clamp(min=0)
    k = torch.where(there[..., None, None], s["k_pool"][page, :, pos % PAGE].float(), 0.0)             # [B][M][Hkv][D]
    bit = torch.arange(N, device=q.device)
    sees = ((s["anc_mask"][:, :, None] >> bit) & 1).bool()                                           # [B][N][N]
    q = q.view(B, N, Hkv, Hq // Hkv, D) * D ** -0.5
    scores = torch.cat([torch.einsum("bngxd,bmgd->bgxnm", q, k),
                        torch.einsum("bngxd,bmgd->bgxnm", q, s["k_tree"].float())], -1)
    del k
    M = pos.numel()
    ok = torch.cat([there[:, None].expand(B, N, M), sees], -1)[:, None, None]
    scores = torch.where(ok, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    del scores
    total = p.sum(-1)                                                                                # [B][Hkv][G][N]
    v = torch.where(there[..., None, None], s["v_pool"][page, :, pos % PAGE].float(), 0.0)
    out = torch.einsum("bgxnm,bmgd->bngxd", p[..., :M], v) + \
        torch.einsum("bgxnm,bmgd->bngxd", p[..., M:], s["v_tree"].float())
    out = out / total.permute(0, 3, 1, 2)[..., None]
    lse = (top[..., 0] + torch.log(total)).permute(0, 3, 1, 2)
    return out.reshape(B, N, Hq, D).to(s["q"].dtype), lse.reshape(B, N, Hq)


def run(state):
    if own:
        return _own(state)
    return globals()["_plain_" + state["op"]](state)


# ------------------------------------------------------------------ what cannot be done without

def work(case):
    """Means of the lengths where they are ragged."""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rope":
        tokens = case["B"] * case["N"]
        return {"bytes": tokens * (4 * (Hq + 2 * Hkv) * D + 8) + 4 * case["B"] + 4 * case["rot"],
                "flops": 3.0 * tokens * (Hq + Hkv) * case["rot"]}
    if case["op"] == "append":
        tokens = case["B"] * case["new"] * (0.75 if case["ragged"] else 1.0)
        k_out = D + 1 if "kq" in case["store"] else 2 * D
        v_out = D + 1 if "v8" in case["store"] else D / 2 + 1 if "v4" in case["store"] else 2 * D
        return {"bytes": tokens * (2 * (Hq + 2 * Hkv) * D + 2 * Hq * D + Hkv * (k_out + v_out)) + 12 * case["B"]
                + tokens / 16 + 4 * case["rot"], "flops": 3.0 * tokens * (Hq + Hkv) * case["rot"]}
    B, N, groups = case["B"], case["N"], case["groups"]
    prefix = case["prefix"] * (0.75 if groups > 1 else 1.0)
    own_keys = case["private"] / 2
    rows = B * N * Hq
    return {"bytes": 4 * Hkv * D * (groups * prefix + B * own_keys) + rows * (4 * D + 4) + B * N * (4 * Hkv * D + 8),
            "flops": 4.0 * rows * D * (prefix + own_keys + 1)}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_turns(r):
    """The rotation of one position, as complex numbers of the pairs' angles, with numpy."""
    rot, factor, out = r["rot"], r["factor"], []
    base = BASE * factor ** (rot / (rot - 2)) if r["scaling"] == "ntk" else BASE
    edges = [rot / 2 * math.log(ORIG / (n * 2 * math.pi), BASE) for n in (FAST, SLOW)]
    for i in range(rot // 2):
        f = 1.0 / base ** (2 * i / rot)
        if r["scaling"] == "linear":
            f /= factor
        if r["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > ORIG / LOW:
                f /= factor
            elif wave >= ORIG / HIGH:
                mix = (ORIG / wave - LOW) / (HIGH - LOW)
                f = (1 - mix) * f / factor + mix * f
        if r["scaling"] == "yarn":
            lo, hi = max(math.floor(edges[0]), 0), min(math.ceil(edges[1]), rot - 1)
            far = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - far) + f / factor * far
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device="cuda"), 1 + 0.1 * math.log(factor) if r["scaling"] == "yarn" else 1.0


def _exact_rotated(x, pos, case):
    f, m = _exact_turns({k: case[k] for k in ("rot", "layout", "scaling", "factor")})
    turn = torch.polar(torch.full_like(pos[..., None] * f, m), pos[..., None] * f)[..., None, :]
    y, rot = x.double().clone(), case["rot"]
    if case["layout"] == "half":
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    return y


def _exact_rope(case, seed):
    s = _prepare_rope(case, seed)
    masks, L = s["anc_mask"].cpu().numpy().view(np.uint64), s["ctx_len"].cpu().numpy()
    pos = [[int(L[b]) + bin(int(m)).count("1") - 1 for m in masks[b]] for b in range(len(L))]
    pos = torch.tensor(pos, dtype=torch.float64, device="cuda")
    return _exact_rotated(s["q"], pos, case), _exact_rotated(s["k"], pos, case), s["v"].double()


def _exact_rows(x, most, bits):
    """Rows as their codes' values: `bits` of mantissa after the leading one (0: whole numbers)."""
    _, e = torch.frexp(x.abs().amax(-1, keepdim=True) / most)
    unit = torch.exp2(e.double())
    unit = torch.where(x.abs().amax(-1, keepdim=True) / most == unit / 2, unit / 2, unit)  # the smallest 2^e >= max / most
    y = x / unit
    if bits:
        _, e = torch.frexp(y)
        step = torch.exp2((e - 1).clamp(min=-6).double() - bits)
    else:
        step = torch.ones_like(y)
    return torch.round(y / step) * step * unit


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    start, L, table = (s[k].cpu().numpy() for k in ("start", "ctx_len", "page_table"))
    seq = np.concatenate([np.full(start[b + 1] - start[b], b) for b in range(len(L))])
    pos = np.concatenate([L[b] + np.arange(start[b + 1] - start[b]) for b in range(len(L))])
    at = torch.from_numpy(table[seq, pos // PAGE].astype(np.int64)).cuda(), torch.from_numpy(pos % PAGE).cuda()
    pos = torch.from_numpy(pos.astype(np.float64)).cuda()
    q, k, v = _exact_rotated(s["q"], pos, case), _exact_rotated(s["k"], pos, case), s["v"].double()
    if "kq" in case["store"]:
        k = _exact_rows(k, 448.0, 3)
    if "v" in case["store"]:
        v = _exact_rows(v, 127.0 if "v8" in case["store"] else 7.0, 0)
    pools = []
    for old, rows in zip(_values(s), (k, v)):
        pool = old.double()
        pool[at[0], :, at[1]] = rows
        pools.append(pool)
    return q, *pools, (L + start[1:] - start[:-1]).astype(np.int32)


def _exact_shared(case, seed):
    s = _prepare_shared(case, seed)
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    out = torch.empty(B, N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, N, Hq, dtype=torch.float64, device="cuda")
    masks = s["anc_mask"].cpu().numpy().view(np.uint64)
    for b in range(B):
        L = int(s["ctx_len"][b])
        at = torch.arange(L, device="cuda")
        page = s["page_table"][b][at // PAGE].long()
        hidden = np.zeros((N, L + N), bool)
        for i in range(N):
            hidden[i, L:] = [not (int(masks[b, i]) >> j) & 1 for j in range(N)]
        hidden = torch.from_numpy(hidden).cuda()
        for g in range(Hkv):
            k = torch.cat([s["k_pool"][page, g, at % PAGE], s["k_tree"][b, :, g]]).double()
            v = torch.cat([s["v_pool"][page, g, at % PAGE], s["v_tree"][b, :, g]]).double()
            hs = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            t = (s["q"][b, :, hs].double() @ k.T / D ** 0.5).masked_fill(hidden[:, None], float("-inf"))
            lse[b, :, hs] = torch.logsumexp(t, -1)
            out[b, :, hs] = torch.exp(t - lse[b, :, hs, None]) @ v
    return out, lse


def exact(case, seed):
    return globals()["_exact_" + case["op"]](case, seed)
