"""Batches in which groups of sequences have their first pages in common, for the tests of the shared-prefix plan and
attention: inputs, and a plan's pieces read back."""
import numpy as np
import torch

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ROWS_MAX, MAX_PARTS = 144, 4


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


def row_groups(N, G):
    NG = max(1, -(-N * G // ROWS_MAX))
    NPG = -(-N // NG)
    while NPG * G > ROWS_MAX and NPG > 1:
        NG += 1
        NPG = -(-N // NG)
    return -(-N // NPG), NPG


def read_plan(plan, B, N, Hq, Hkv, D, groups):
    """A plan's parts as arrays of 32-bit words."""
    raw = plan.cpu().numpy().tobytes()
    head = np.frombuffer(raw, np.int32, 16)
    C, G = int(head[7]), Hq // Hkv
    NG, NPG = row_groups(N, G)
    nodes = -(-B // groups) * N
    blocks = -(-nodes // (ROWS_MAX // G))
    block = -(-nodes // blocks)
    sizes = dict(head=(1, 16), cta=(C, 4), grp=(groups, 4), seq=(B, 5), seg=(B * Hkv * NG, 2), lcp=(B, 1),
                 item=(MAX_PARTS * C + Hkv * (B * N // block + groups), 12), piece=(C + B * Hkv * NG, 12))
    at, out = 0, dict(NG=NG, NPG=NPG, block=block, C=C)
    for name, (n, w) in sizes.items():
        out[name] = np.frombuffer(raw, np.int32, n * w, at).reshape(n, w)
        at += -(-4 * n * w // 16) * 16
    assert at == len(raw)
    return out


def check_plan(plan, ctx, start, table, pages, N, Hq, Hkv, D):
    """Every tile of every segment belongs to exactly one piece of one CTA, and every number is in its range."""
    B, groups = len(ctx), len(start) - 1
    p = read_plan(plan, B, N, Hq, Hkv, D, groups)
    C, NG, NPG, block = p["C"], p["NG"], p["NPG"], p["block"]
    assert list(p["head"][0, 1:10]) == [B, N, Hq, Hkv, D, groups, C, table.shape[1], pages]
    items = int(p["head"][0, 10])
    assert items <= len(p["item"])
    both = common(ctx, start, table, pages)
    used = p["grp"][:, 0]
    assert all(u in (0, n) for u, n in zip(used, both))
    seen_item, seen_own, tiles_done, own_done = set(), set(), {}, {}
    for c in range(C):
        own0, owns, tiles, its = p["cta"][c]
        total = 0
        for k in range(its):
            i = c + k * C
            assert i < items and i not in seen_item
            seen_item.add(i)
            b, g, node0, nodes, page0, vp, ta, te, keys, slot, own, reread = p["item"][i]
            grp = list(start).index(b, 0) if start.tolist().count(b) == 1 else max(x for x in range(groups) if start[x] == b)
            z = start[grp + 1]
            assert own == 0 and slot == i and page0 == 0 and vp == used[grp] > 0 and keys == vp * PAGE and 0 <= g < Hkv
            assert 0 <= ta < te <= (vp + 1) // 2 and (node0 - b * N) % block == 0
            assert 1 <= nodes <= block and node0 + nodes <= z * N and (nodes == block or node0 + nodes == z * N)
            assert i == p["grp"][grp, 1] + (g * p["grp"][grp, 2] + part_of(ta, (vp + 1) // 2, p["grp"][grp, 2])) * \
                p["grp"][grp, 3] + (node0 - b * N) // block
            tiles_done.setdefault((grp, g, node0), []).append((ta, te))
            total += te - ta
        for k in range(owns):
            i = own0 + k
            assert 0 <= i < len(p["piece"]) and i not in seen_own
            seen_own.add(i)
            b, g, node0, nodes, page0, vp, ta, te, keys, slot, own, reread = p["piece"][i]
            grp = max(x for x in range(groups) if start[x] <= b)
            u = used[grp]
            assert own == 1 and 0 <= b < B and 0 <= g < Hkv and page0 == u and vp == -(-int(ctx[b]) // PAGE) - u >= 0
            assert keys == ctx[b] - u * PAGE >= 0 and (node0 - b * N) % NPG == 0
            rg = (node0 - b * N) // NPG
            assert 0 <= rg < NG and nodes == min(NPG, N - rg * NPG) and 0 <= ta < te <= (vp + 2) // 2
            s = (b * Hkv + g) * NG + rg
            first, count = p["seg"][s]
            whole = (ta, te) == (0, (vp + 2) // 2) and u == 0
            assert (slot == -1) == whole == (count < 0)
            if not whole:
                assert slot == i and first <= i < first + count
            own_done.setdefault(s, []).append((ta, te))
            total += te - ta
        assert total == tiles
    assert seen_item == set(range(items))
    for g in range(groups):
        n = (start[g + 1] - start[g]) * N
        if used[g]:
            for h in range(Hkv):
                for x in range(-(-n // block)):
                    joins(tiles_done.pop((g, h, start[g] * N + x * block)), (used[g] + 1) // 2)
    assert not tiles_done
    for s in range(B * Hkv * NG):
        b = s // (Hkv * NG)
        u = used[max(x for x in range(groups) if start[x] <= b)]
        joins(own_done[s], (-(-int(ctx[b]) // PAGE) - u + 2) // 2)
        if p["seg"][s, 1] > 0:
            assert p["seg"][s, 1] == len(own_done[s])
    return p


def part_of(ta, tiles, parts):
    return next(j for j in range(parts) if tiles * j // parts == ta)


def joins(ranges, tiles):
    at = 0
    for a, z in sorted(ranges):
        assert a == at < z
        at = z
    assert at == tiles
