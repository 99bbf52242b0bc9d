"""Rotary positions and appends to the paged cache against the formulas in 64 bits: both layouts, parts of the head,
far and negative positions, strided views, sequences of no, one and many new tokens, every pool format, pages that are
missing."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
KQ, V8, V4 = "e4m3", "int8", "int4"


def _lt():
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    return LT


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def projection(lead, Hq, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*lead, (Hq + 2 * Hkv) * D, generator=g).to(TYPES[dtype]).cuda()
    return tuple(t.unflatten(-1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], -1))


def rotated(x, pos, rot, layout, base=10000.0, magnitude=1.0):
    """(x rotated, how far a correct kernel may be from it before its rounding): x [rows][H][D], pos [rows].

    The angle's fraction of a turn is exact to 2^-32, in fp32 to 2^-25 of a half turn (9.4e-8 rad); sincospif is
    within 2^-22 of a value of at most 1, three products and sums round by 2^-24 each: less than 2^-21 of
    m (|x| + |y|) together.  The reference's own angle, p f in 64 bits, is off by 2^-51 p f."""
    x, pos = x.double().cpu(), pos.double().cpu()
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = pos[:, None] * f
    c, s = torch.cos(a)[:, None] * magnitude, torch.sin(a)[:, None] * magnitude
    lost = (2.0 ** -21 + 2.0 ** -51 * a.abs())[:, None] * magnitude
    y, err = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2)
    i, j = (i, i + rot // 2) if layout == 0 else (2 * i, 2 * i + 1)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    err[..., i] = err[..., j] = (x[..., i].abs() + x[..., j].abs()) * lost
    return y, err


def near(got, want, err):
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * half  # half a step of the subnormal ones
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    bound = err + half * (want.abs() + err) + tiny
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())


#        B, N, Hq, Hkv, D,  rot, layout, dtype
ROPE = [
    (1, 8, 8, 2, 128, 128, 0, "f16"), (3, 22, 24, 4, 256, 64, 0, "bf16"), (2, 5, 6, 3, 256, 256, 1, "bf16"),
    (1, 1, 1, 1, 16, 2, 0, "f16"), (1, 1, 1, 1, 16, 2, 1, "f16"), (2, 3, 5, 5, 96, 96, 0, "bf16"),
    (2, 7, 3, 1, 80, 20, 0, "f16"), (2, 7, 3, 1, 80, 20, 1, "f16"), (1, 64, 15, 5, 128, 100, 0, "bf16"),
    (4, 16, 2, 1, 1024, 1024, 0, "bf16"), (1, 3, 33, 11, 272, 250, 0, "f16"), (300, 2, 2, 2, 64, 64, 1, "f16"),
    (64, 64, 16, 4, 128, 128, 0, "bf16"),
]


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_tree_positions(cuda_dev, case):
    B, N, Hq, Hkv, D, rot, layout, dtype = case
    LT, rng = _lt(), np.random.default_rng(sum(case[:6]))
    q, k, v = projection((B, N), Hq, Hkv, D, dtype, B + N)
    parent = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        parent[:, i] = rng.integers(-1, i, size=B)
    depth = np.zeros((B, N), np.int64)
    for i in range(N):
        depth[:, i] = np.where(parent[:, i] < 0, 0, depth[np.arange(B), parent[:, i]] + 1)
    status, anc = _status(), torch.empty(B, N, dtype=torch.int64, device="cuda")
    LT.lucetree_build_anc_mask(torch.from_numpy(parent).cuda(), anc, status)
    ctx = rng.integers(0, 200000, size=B)
    steps, m = LT.lucetree_rope_steps(rot, 10000.0)
    out = [torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda") for t in (q, k, v)]
    LT.lucetree_rope(q, k, steps.cuda(), layout, out[0], out[1], status, v=v, v_out=out[2], magnitude=1.25,
                     ctx_len=torch.from_numpy(ctx.astype(np.int32)).cuda(), anc_mask=anc)
    assert int(status.item()) == 0
    pos = torch.from_numpy(ctx[:, None] + depth).flatten()
    for x, y in zip((q, k), out):
        near(y.flatten(0, 1), *rotated(x.flatten(0, 1), pos, rot, layout, magnitude=1.25))
        assert torch.equal(y[..., rot:], x[..., rot:])
    assert torch.equal(out[2], v)


def test_any_position(cuda_dev):
    LT = _lt()
    pos = [0, 1, -1, 63, 131071, 10 ** 6 + 1, -(10 ** 6), 2 ** 31 - 1, -2 ** 31, 12345678, 2 ** 30]
    N = len(pos)
    q, k, _ = projection((1, N), 3, 1, 128, "f16", 5)
    p = torch.tensor([pos], dtype=torch.int32, device="cuda")
    for layout in (0, 1):
        steps, _ = LT.lucetree_rope_steps(128, 10000.0)
        out, status = (torch.empty(1, N, 3, 128, dtype=torch.float16, device="cuda"),
                       torch.empty(1, N, 1, 128, dtype=torch.float16, device="cuda")), _status()
        LT.lucetree_rope(q, k, steps.cuda(), layout, *out, status, positions=p)
        near(out[0][0], *rotated(q[0], p[0], 128, layout))
        near(out[1][0], *rotated(k[0], p[0], 128, layout))


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("magnitude", [1.0, 1.1386294])
def test_cosines_within_a_step(cuda_dev, layout, magnitude):
    """A cosine is off by less than a step of fp32 (2^-23 m), the product that is rounded apart and the sum by half a
    step each: less than 2^-22 of m (|x| + |y|) together."""
    LT, N = _lt(), 3000
    q, k, _ = projection((1, N), 2, 1, 256, "f16", 8)
    pos = torch.randint(0, 2 ** 20, (1, N), generator=torch.Generator().manual_seed(4), dtype=torch.int32)
    pos[0, :5] = torch.tensor([0, 1, 2, 2 ** 20, 2 ** 31 - 1])
    steps, _ = LT.lucetree_rope_steps(256, 10000.0)
    out, status = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)], _status()
    LT.lucetree_rope(q, k, steps.cuda(), layout, *out, status, positions=pos.cuda(), magnitude=magnitude)
    m = float(np.float32(magnitude))
    for x, y in zip((q, k), out):
        want, err = rotated(x[0], pos[0], 256, layout, magnitude=m)
        near(y[0], want, err * (2.0 ** -22 / 2.0 ** -21))


def test_scores_depend_on_distance_alone(cuda_dev):
    """q at p + d and k at p have the same product for every p: the angles of far positions are as exact as near ones."""
    LT = _lt()
    g = torch.Generator().manual_seed(3)
    x, y = torch.randn(256, generator=g).half(), torch.randn(256, generator=g).half()
    base = torch.tensor([0, 5, 1000, 131072, 10 ** 7], dtype=torch.int32)
    n = len(base)
    q, k = x.expand(1, n, 1, 256).contiguous().cuda(), y.expand(1, n, 1, 256).contiguous().cuda()
    steps, _ = LT.lucetree_rope_steps(256, 1e6)
    steps = steps.cuda()
    outs = []
    for pos in (base + 17, base):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        LT.lucetree_rope(q, k, steps, 0, qo, ko, _status(), positions=pos[None].cuda())
        outs.append((qo if pos is not base else ko)[0, :, 0].double().cpu())
    s = (outs[0] * outs[1]).sum(-1)
    # each rotated value is rounded to fp16 (2^-11 of it) and off by 2^-21 of its pair's magnitudes
    room = (outs[0].abs() * outs[1].abs()).sum(-1).max() * 2 * 2 * (2.0 ** -11 + 2.0 ** -19)
    assert (s - s[0]).abs().max() <= room


def test_masks_and_lengths_that_are_bad_are_flagged(cuda_dev):
    LT = _lt()
    q, k, _ = projection((2, 2), 2, 1, 32, "f16", 1)
    steps = LT.lucetree_rope_steps(32, 1e4)[0].cuda()
    out = torch.empty(2, 2, 2, 32, dtype=torch.float16, device="cuda"), torch.empty(2, 2, 1, 32, dtype=torch.float16, device="cuda")
    status = _status()
    anc = torch.tensor([[1, 1], [1, 3]], dtype=torch.int64, device="cuda")  # node 1 of sequence 0 lacks itself
    LT.lucetree_rope(q, k, steps, 0, *out, status, ctx_len=torch.tensor([7, -3], dtype=torch.int32, device="cuda"), anc_mask=anc)
    assert int(status.item()) == LT.DEV_BAD_NODE | LT.DEV_BAD_CTX
    near(out[0].flatten(0, 1), *rotated(q.flatten(0, 1), torch.tensor([7, 7, 0, 1]), 32, 0))


# ------------------------------------------------------------------ appends

def e4m3_codes(x):
    """Codes and exponents of rows x [..., D] of 64-bit values, and the largest values' exponents p."""
    m = x.abs().amax(-1)
    p = torch.floor(torch.log2(448 / m))
    p = torch.where(m * 2.0 ** p > 448, p - 1, torch.where(m * 2.0 ** (p + 1) <= 448, p + 1, p))
    return p


def int_rows(v, most):
    """Values that v [.., D] (16-bit) is stored as."""
    v = v.double().cpu()
    m = v.abs().amax(-1, keepdim=True)
    p = torch.floor(torch.log2(most / torch.where(m > 0, m, 1.0)))
    p = torch.where(m * 2.0 ** p > most, p - 1, torch.where(m * 2.0 ** (p + 1) <= most, p + 1, p))
    return torch.where((m > 0) & (p <= 126), torch.round(v * 2.0 ** p) * 2.0 ** -p, 0.0)


def values(codes, exps, fmt):
    e = exps.cpu().double()
    scale = torch.where(e > 0, 2.0 ** (e - 127), 0.0)[..., None]
    c = codes.cpu()
    if fmt == KQ:
        return c.view(torch.float8_e4m3fn).double() * scale
    c = c.view(torch.int8)
    if fmt == V4:
        c = torch.stack([(c << 4) >> 4, c >> 4], -1).flatten(-2)
    return c.double() * scale


class Cache:
    def __init__(self, ctx, new, Hkv, D, dtype, kf="same", vf="same", seed=0, spare=2, fill=True):
        rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.kf, self.vf = np.array(ctx), np.array(new), kf, vf
        per = -(-(self.ctx + self.new) // PAGE)
        P = int(per.sum()) + spare
        ids = rng.permutation(P)
        self.table = np.full((len(ctx), max(1, int(per.max()))), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.pools, self.exps = [], []
        for fmt in (kf, vf):
            if fmt == "same":
                self.pools.append(torch.randn(P, Hkv, PAGE, D, generator=g).to(TYPES[dtype]).cuda())
                self.exps.append(None)
            else:
                self.pools.append(torch.randint(0, 120, (P, Hkv, PAGE, D // 2 if fmt == V4 else D), generator=g,
                                                dtype=torch.uint8).cuda())
                self.exps.append(torch.randint(1, 250, (P, Hkv, PAGE), generator=g, dtype=torch.uint8).cuda())

    def places(self, b):
        pos = np.arange(self.ctx[b], self.ctx[b] + self.new[b])
        return self.table[b, pos // PAGE], pos % PAGE

    def append(self, q, k, v, start, steps=None, layout=0, magnitude=1.0, table=None, ctx=None, stream=None):
        LT = _lt()
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.ctx_out = torch.full((len(self.ctx),), -7, dtype=torch.int32, device="cuda")
        self.q_out = None if q is None else torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        self.status = _status()
        vf = {"same": LT.LUCETREE_V_SAME, V8: LT.LUCETREE_V_INT8, V4: LT.LUCETREE_V_INT4}[self.vf]
        LT.lucetree_append_kv(k, v, i32(start), i32(self.table if table is None else table), i32(self.ctx if ctx is None else ctx),
                              self.ctx_out, self.pools[0], self.pools[1], self.status, q=q, q_out=self.q_out, steps=steps,
                              layout=layout, magnitude=magnitude, k_exp=self.exps[0], v_format=vf, v_exp=self.exps[1],
                              stream=stream)
        torch.cuda.synchronize()
        return int(self.status.item())


def check_append(ctx, new, Hq, Hkv, D, dtype, rot, layout, kf="same", vf="same", gap=0, seed=0):
    """gap: rows before the first sequence's and after the last one's that belong to none."""
    LT = _lt()
    c = Cache(ctx, new, Hkv, D, dtype, kf, vf, seed)
    start = gap + np.concatenate([[0], np.cumsum(c.new)])
    T = int(start[-1]) + gap
    q, k, v = projection((T,), max(Hq, 1), Hkv, D, dtype, seed + 1)
    before = [(None if t is None else t.clone()) for t in c.pools + c.exps]
    steps = LT.lucetree_rope_steps(rot, 10000.0)[0].cuda() if rot else None
    assert c.append(q if Hq else None, k, v, start, steps, layout, 0.75 if rot else 1.0) == 0
    assert np.array_equal(c.ctx_out.cpu().numpy(), c.ctx + c.new)
    pos = np.concatenate([L + np.arange(n) for L, n in zip(c.ctx, c.new)] + [np.zeros(0)])
    mine = slice(gap, T - gap)
    turn = (lambda x: rotated(x[mine], torch.from_numpy(pos), rot, layout, magnitude=0.75)) if rot else \
        (lambda x: (x[mine].double().cpu(), torch.zeros(x[mine].shape, dtype=torch.float64)))
    if Hq:
        near(c.q_out[mine], *turn(q))
        assert (c.q_out[:gap] == 7).all() and (c.q_out[T - gap:] == 7).all()
    page = torch.from_numpy(np.concatenate([c.places(b)[0] for b in range(len(ctx))]).astype(np.int64))
    slot = torch.from_numpy(np.concatenate([c.places(b)[1] for b in range(len(ctx))]).astype(np.int64))
    kw, kerr = turn(k)
    if kf == "same":
        near(c.pools[0].cpu()[page, :, slot], kw, kerr)
    else:
        got, e = values(c.pools[0], c.exps[0], KQ)[page, :, slot], c.exps[0].cpu().double()[page, :, slot]
        # the exponent of a row whose largest value lies next to 448 2^-p may be the neighbour's
        assert ((127 - e == e4m3_codes(kw * (1 - 2.0 ** -19))) | (127 - e == e4m3_codes(kw * (1 + 2.0 ** -19)))).all()
        # half a step: 2^-4 of a value, or 2^-10 (of 2^-9 steps) below the smallest normal one
        bound = kerr + 2.0 ** -4 * (kw.abs() + kerr) + 2.0 ** -10 * 2.0 ** (e - 127)[..., None]
        assert ((got - kw).abs() <= bound).all()
    vw = v[mine].double().cpu()
    if vf == "same":
        assert torch.equal(c.pools[1].cpu()[page, :, slot].double(), vw)
    else:
        assert torch.equal(values(c.pools[1], c.exps[1], vf)[page, :, slot], int_rows(v[mine], 127.0 if vf == V8 else 7.0))
    # every other byte is as it was
    for was, now in zip(before, c.pools + c.exps):
        if was is not None:
            now = now.clone()
            now[page.cuda(), :, slot.cuda()] = was[page.cuda(), :, slot.cuda()]
            assert torch.equal(now.view(torch.uint8), was.view(torch.uint8))
    return c


#         ctx,                    new,                   Hq, Hkv, D,  dtype, rot, layout
APPEND = [
    ((1000,),                    (1,),                    24, 4, 256, "bf16", 256, 0),
    ((0, 1, 63, 64, 65, 127),    (0, 1, 1, 1, 64, 129),    8, 2, 128, "f16",  128, 1),
    ((5, 0, 0),                  (0, 0, 0),                4, 2, 128, "f16",  64,  0),
    ((0,),                       (1000,),                  6, 6, 64,  "bf16", 32,  0),
    ((300, 7),                   (100, 333),              15, 5, 128, "f16",  96,  1),
    ((62, 63, 64),               (3, 66, 130),             4, 2, 80,  "bf16", 20,  0),
    ((9,) * 40,                  (1,) * 40,                8, 2, 256, "bf16", 64,  0),
    ((100, 3),                   (5, 70),                  0, 3, 128, "f16",  128, 0),
    ((100, 3),                   (5, 70),                  4, 2, 128, "f16",  0,   0),
    ((0, 10),                    (3000, 1100),             4, 1, 16,  "bf16", 16,  0),
]


@pytest.mark.parametrize("gap", [0, 3])
@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(cuda_dev, case, gap):
    check_append(*case, gap=gap, seed=len(case[0]) + case[4])


def test_append_many_sequences(cuda_dev):
    rng = np.random.default_rng(2)
    B = 700
    check_append(tuple(rng.integers(0, 300, B)), tuple(rng.integers(0, 4, B)), 2, 1, 64, "bf16", 64, 0, gap=1)


@pytest.mark.parametrize("kf,vf", [("same", V8), ("same", V4), (KQ, "same"), (KQ, V8), (KQ, V4)])
@pytest.mark.parametrize("rot,layout", [(256, 0), (64, 1), (0, 0), (100, 0)])
def test_append_codes(cuda_dev, kf, vf, rot, layout):
    check_append((0, 61, 200, 8), (70, 5, 1, 0), 6, 3, 256, "bf16", rot, layout, kf, vf, gap=2, seed=rot)
    if kf == "same":
        check_append((3,), (300,), 0, 1, 256, "f16", rot, layout, kf, vf, seed=rot)


def test_rows_of_zeros_and_of_tiny_values_as_codes(cuda_dev):
    c = Cache((0,), (4,), 2, 256, "bf16", KQ, V8)
    k = torch.zeros(4, 2, 256, dtype=torch.bfloat16, device="cuda")
    k[1] = 2.0 ** -125     # its exponent byte would leave [1, 254]
    k[2] = 2.0 ** -100
    k[3, 0, 7] = -3e38
    assert c.append(None, k, k.clone(), [0, 4]) == 0
    page = int(c.table[0, 0])
    got = values(c.pools[0], c.exps[0], KQ)[page, :, :4].transpose(0, 1)
    want = k.double().cpu()
    want[1] = 0
    assert torch.equal(got[:3], want[:3])
    assert abs(got[3, 0, 7] / want[3, 0, 7] - 1) <= 2.0 ** -4 and (got[3, 1] == 0).all()
    assert (c.exps[0][page, :, 0] == 0).all() and (c.exps[1][page, :, :2] == 0).all()
    got = values(c.pools[1], c.exps[1], V8)[page, :, :4].transpose(0, 1)
    assert torch.equal(got[:3], want[:3]) and abs(got[3, 0, 7] / want[3, 0, 7] - 1) <= 1 / 127


def test_append_equals_rotation_and_commit(cuda_dev):
    """A chain of accepted nodes, rotated and committed, and the same tokens appended: the same pools, bit for bit."""
    LT = _lt()
    B, N, Hq, Hkv, D = 3, 7, 4, 2, 256
    ctx = (60, 0, 129)
    q, k, v = projection((B, N), Hq, Hkv, D, "bf16", 8)
    steps = LT.lucetree_rope_steps(D, 1e4)[0].cuda()
    a = Cache(ctx, (N,) * B, Hkv, D, "bf16", seed=4)
    b = Cache(ctx, (N,) * B, Hkv, D, "bf16", seed=4)
    assert a.append(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), np.arange(B + 1) * N, steps) == 0
    chain = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    status, anc = _status(), torch.empty(B, N, dtype=torch.int64, device="cuda")
    LT.lucetree_build_anc_mask(chain - 1, anc, status)
    L = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    out = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k, v)]
    LT.lucetree_rope(q, k, steps, 0, out[0], out[1], status, ctx_len=L, anc_mask=anc, v=v, v_out=out[2])
    ctx_out = torch.empty_like(L)
    LT.lucetree_commit(out[1], out[2], chain, torch.full((B,), N, dtype=torch.int32, device="cuda"),
                       torch.from_numpy(b.table).cuda(), L, ctx_out, b.pools[0], b.pools[1], status)
    assert int(status.item()) == 0 and torch.equal(a.ctx_out, ctx_out)
    assert torch.equal(a.q_out, out[0].flatten(0, 1))
    for x, y in zip(a.pools, b.pools):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_unrotated_codes_equal_the_commit_of_codes(cuda_dev):
    LT = _lt()
    N, Hkv = 9, 3
    _, k, v = projection((1, N), 1, Hkv, 256, "bf16", 11)
    a, b = (Cache((60,), (N,), Hkv, 256, "bf16", KQ, "same", seed=6) for _ in range(2))
    assert a.append(None, k[0], v[0], [0, N]) == 0
    status, L = _status(), torch.tensor([60], dtype=torch.int32, device="cuda")
    LT.lucetree_commit_kq(k.contiguous(), v.contiguous(), torch.arange(N, dtype=torch.int32, device="cuda")[None].contiguous(),
                          torch.tensor([N], dtype=torch.int32, device="cuda"), torch.from_numpy(b.table).cuda(), L,
                          torch.empty_like(L), b.pools[0], b.exps[0], b.pools[1], status)
    assert torch.equal(a.pools[0], b.pools[0]) and torch.equal(a.exps[0], b.exps[0])


def test_missing_pages_end_the_length(cuda_dev):
    LT = _lt()
    q, k, v = projection((300,), 2, 1, 64, "f16", 3)
    c = Cache((10, 60, 0), (200, 50, 50), 1, 64, "f16")
    table = c.table.copy()
    table[0, 2] = c.pools[0].shape[0]  # positions 128 .. 191 of sequence 0
    table[1, 1] = -1                   # positions 64 .. of sequence 1
    was = [p.clone() for p in c.pools]
    assert c.append(q, k, v, [0, 200, 250, 300], None, table=table) == LT.DEV_BAD_PAGE
    assert c.ctx_out.tolist() == [128, 64, 50]
    assert torch.equal(c.q_out, q)  # queries have a position all the same
    for pool, old, x in zip(c.pools, was, (k, v)):
        for b, s, n in ((0, 0, 118), (1, 200, 4), (2, 250, 50)):
            page, slot = (torch.from_numpy(t[:n].astype(np.int64)).cuda() for t in c.places(b))
            assert torch.equal(pool[page, :, slot], x[s:s + n])
        for page in (c.table[0, 2], c.table[1, 1]):
            assert torch.equal(pool[int(page)], old[int(page)])


@pytest.mark.parametrize("start", [(0, 5, 3), (-1, 2, 4), (0, 2, 99), (3, 2, 4)])
def test_bad_starts_append_nothing(cuda_dev, start):
    LT = _lt()
    q, k, v = projection((6,), 2, 1, 64, "f16", 3)
    c = Cache((10, 60), (6, 6), 1, 64, "f16")
    was = [p.clone() for p in c.pools]
    assert c.append(q, k, v, start, None) == LT.DEV_BAD_ROW
    assert c.ctx_out.tolist() == [10, 60] and (c.q_out == 7).all()
    assert all(torch.equal(a, b) for a, b in zip(was, c.pools))


def test_bad_lengths_append_nothing_to_their_sequence(cuda_dev):
    LT = _lt()
    q, k, v = projection((9,), 2, 1, 64, "f16", 3)
    c = Cache((10, 60, 5), (3, 3, 3), 1, 64, "f16")
    assert c.append(q, k, v, [0, 3, 6, 9], None, ctx=[10, -4, 1000]) == LT.DEV_BAD_CTX
    assert c.ctx_out.tolist() == [13, -4, 1000]
    assert torch.equal(c.q_out[:3], q[:3]) and (c.q_out[3:] == 7).all()


def test_a_table_that_ends_inside_the_new_tokens(cuda_dev):
    LT = _lt()
    q, k, v = projection((100,), 2, 1, 64, "f16", 3)
    c = Cache((50,), (100,), 1, 64, "f16")
    assert c.append(q, k, v, [0, 100], None, table=c.table[:, :2]) == LT.DEV_BAD_PAGE
    assert c.ctx_out.tolist() == [128]


def test_captured_and_on_another_stream(cuda_dev):
    LT = _lt()
    q, k, v = projection((4,), 2, 1, 128, "bf16", 3)
    c = Cache((62, 5), (2, 2), 1, 128, "bf16")
    steps = LT.lucetree_rope_steps(128, 1e4)[0].cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert c.append(q, k, v, [0, 2, 4], steps, stream=side) == 0
    want = [c.q_out.clone(), *(p.clone() for p in c.pools)]
    d = Cache((62, 5), (2, 2), 1, 128, "bf16")
    start, table, L = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2, 4], d.table.tolist(), [62, 5]))
    q2, k2, v2 = (torch.zeros_like(t.contiguous()) for t in (q, k, v))
    qo, lo, status = torch.empty_like(q2), torch.empty_like(L), _status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        LT.lucetree_append_kv(k2, v2, start, table, L, lo, d.pools[0], d.pools[1], status, q=q2, q_out=qo, steps=steps)
    for a, b in ((q2, q), (k2, k), (v2, v)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and lo.tolist() == [64, 7]
    for x, y in zip(want, [qo, *d.pools]):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_pools_past_four_gigabytes(cuda_dev):
    LT = _lt()
    pages = 70000  # 70,000 pages of 64 KB
    _, k, v = projection((3,), 1, 4, 128, "bf16", 3)
    pools = [torch.zeros(pages, 4, PAGE, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    lo, status = i32(0), _status()
    LT.lucetree_append_kv(k, v, i32(0, 3), i32(pages - 1, 3)[None].contiguous(), i32(62), lo, *pools, status)
    assert int(status.item()) == 0 and int(lo.item()) == 65
    for pool, x in zip(pools, (k, v)):
        assert torch.equal(pool[pages - 1, :, 62:].transpose(0, 1), x[:2]) and torch.equal(pool[3, :, 0], x[2])
        assert int(torch.count_nonzero(pool.view(pages, -1).any(1))) == 2
