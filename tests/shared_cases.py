"""Batches in which groups of sequences have their first pages in common, for the tests of the shared-prefix plan and
attention: inputs, and a plan's pieces read back."""
import numpy as np
import torch

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ROWS = 128


def batch(groups, N, seed=0, spare=3, reserve=0):
    """groups: one (pages in common, lengths of its sequences) after the other.  -> lengths, starts, table, pages."""
    rng = np.random.default_rng(seed)
    ctx = [L for _, Ls in groups for L in Ls]
    start = np.concatenate([[0], np.cumsum([len(Ls) for _, Ls in groups])])
    per = [-(-(L + N) // PAGE) for L in ctx]
    maxp = max(per) + reserve
    table = np.full((len(ctx), maxp), -1, np.int32)
    ids = rng.permutation(sum(per) + spare)
    at = b = 0
    for both, Ls in groups:
        first = b
        for _ in Ls:
            lo = min(both, per[b], per[first]) if b != first else 0
            table[b, :lo] = table[first, :lo]
            table[b, lo:per[b]] = ids[at:at + per[b] - lo]
            at += per[b] - lo
            b += 1
    return np.array(ctx, np.int32), start.astype(np.int32), table, len(ids)


def common(ctx, start, table, pages):
    """Leading pages that the sequences of each group have in common and have filled."""
    out = []
    for a, z in zip(start[:-1], start[1:]):
        n = 0
        while z - a > 1 and n < min(ctx[a:z]) // PAGE and 0 <= table[a, n] < pages and (table[a:z, n] == table[a, n]).all():
            n += 1
        out.append(n)
    return out


def block_nodes(nodes, N, cap):
    blocks = -(-nodes // cap)
    per = -(-nodes // blocks)
    whole = -(-per // N) * N
    if whole <= cap:
        return whole
    if cap >= N and -(-nodes // (cap // N * N)) <= blocks:
        return cap // N * N
    return per


def read_plan(plan, B, N, Hq, Hkv, D, groups):
    """A plan's parts as arrays of 32-bit words."""
    raw = plan.cpu().numpy().tobytes()
    head = np.frombuffer(raw, np.int32, 16)
    G = Hq // Hkv
    pair = 2 if -(-B // groups) * N * G > ROWS else 1
    C, cap = int(head[7]), ROWS // G * pair
    NG = -(-N // cap)
    NPGo = -(-N // NG)
    NG = -(-N // NPGo)
    sizes = dict(head=(1, 16), cta=(C, 4), grp=(groups + 1, 5), seq=(B + 1, 6), blk=(B * NG + 1, 8), split=(C, 8), piece=(C + B * NG * Hkv, 12))
    at, out = 0, dict(NG=NG, NPGo=NPGo, NPG=block_nodes(-(-B // groups) * N, N, cap), C=C, rows=ROWS * pair)
    for name, (n, w) in sizes.items():
        out[name] = np.frombuffer(raw, np.int32, n * w, at).reshape(n, w)
        at += -(-4 * n * w // 16) * 16
    assert at == len(raw)
    return out


def check_plan(plan, ctx, start, table, pages, N, Hq, Hkv, D):
    """Every row is in exactly one block, every page of a block's sequences in its key list, and every tile of every
    segment in exactly one piece of one CTA; the rows of partial sums do not overlap."""
    B, groups, G = len(ctx), len(start) - 1, Hq // Hkv
    p = read_plan(plan, B, N, Hq, Hkv, D, groups)
    C, NG, NPGo, NPG = p["C"], p["NG"], p["NPGo"], p["NPG"]
    assert max(NPG, NPGo) * G <= p["rows"]
    assert list(p["head"][0, 1:10]) == [B, N, Hq, Hkv, D, groups, C, table.shape[1], pages]
    blocks = int(p["head"][0, 10])
    assert blocks <= B * NG
    both, of = common(ctx, start, table, pages), [max(g for g in range(groups) if start[g] <= b) for b in range(B)]
    used = p["grp"][:groups, 0]
    assert all(u in (0, n) for u, n in zip(used, both))
    own = [-(-int(ctx[b]) // PAGE) - used[of[b]] for b in range(B)]
    assert list(p["seq"][:, 4]) == list(np.concatenate([[0], np.cumsum(own)]))
    node = 0
    for k in range(blocks):
        group, b0, seqs, node0, nodes, u, vp, _ = p["blk"][k]
        assert node0 == node and 1 <= nodes <= (NPG if u else NPGo)
        assert b0 == node0 // N and seqs == (node0 + nodes - 1) // N - b0 + 1 and (seqs == 1 or u)
        assert group == of[b0] == of[b0 + seqs - 1] and u == used[group] and vp == u + sum(own[b0:b0 + seqs]) + -(-seqs * N // PAGE)
        node += nodes
    assert node == B * N
    # segments in the flat order: group, KV head, block
    segs = []
    for g in range(groups):
        mine = [k for k in range(blocks) if p["blk"][k, 0] == g]
        segs += [(k, h) for h in range(Hkv) for k in mine]
    done, rows, splits = {}, [], {}
    for c in range(C):
        then, n, tiles, _ = p["cta"][c]
        count = 0
        for s in range(then - 1 - C, then - 1 - C + n):
            i = c if s == then - 1 - C else C + s
            assert 0 <= i < len(p["piece"])
            b0, seqs, node0, nodes, u, vp, ta, te, g, slot, alone, _ = p["piece"][i]
            block = segs[s][0]
            assert list(p["blk"][block, 1:7]) == [b0, seqs, node0, nodes, u, vp] and segs[s][1] == g
            assert 0 <= ta < te <= (vp + 1) // 2 and alone == (u == 0)
            whole = (ta, te) == (0, (vp + 1) // 2)
            assert (slot < 0) == whole
            if not whole:
                rows.append((slot, nodes * G))
                k = c - len(done.get(s, []))  # the CTA that has its first tiles
                n_split, row, n0, n_rows, head = p["split"][k, :5]
                assert (n0, n_rows, head) == (node0, nodes * G, g) and slot == row + p["rows"] * (c - k)
                splits[s] = (k, n_split)
            done.setdefault(s, []).append((ta, te))
            count += te - ta
        assert count == tiles
    for s, (k, _) in enumerate(segs):
        joins(done[s], (p["blk"][k, 6] + 1) // 2)
        assert len(done[s]) == splits.get(s, (0, 1))[1]
    assert sorted(k for k, _ in splits.values()) == list(np.nonzero(p["split"][:, 0])[0])
    at = 0
    for slot, n in sorted(rows):
        assert slot >= at
        at = slot + n
    assert at <= B * N * Hq + p["rows"] * C
    return p


def joins(ranges, tiles):
    at = 0
    for a, z in sorted(ranges):
        assert a == at < z
        at = z
    assert at == tiles
