"""Outputs, plans and workspaces of exactly the sizes that are asked for, between guard bytes that no call may change:
rotation, append, the plan of a shared batch and its attention."""
import numpy as np
import pytest
import torch

from tests.shared_cases import TYPES
from tests.test_gpu_attention_shared import P_STEP, _lt, make, near, reference
from tests.test_gpu_shared_uneven import fork

pytestmark = pytest.mark.gpu

GUARD, FILL = 4096, 0x5A


class Guarded:
    """Buffers between guard bytes."""

    def __init__(self):
        self.all = []

    def take(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((GUARD + n + GUARD,), FILL, dtype=torch.uint8, device="cuda")
        assert raw.data_ptr() % 256 == 0
        self.all.append((raw, n))
        return raw[GUARD:GUARD + n].view(dtype).view(shape)

    def untouched(self):
        torch.cuda.synchronize()
        return all(bool((raw[:GUARD] == FILL).all()) and bool((raw[GUARD + n:] == FILL).all()) for raw, n in self.all)


def test_guards_see_a_byte(cuda_dev):
    for at in (-1, 12):
        g = Guarded()
        g.take((3,), torch.int32)
        g.all[0][0][GUARD + at] = 0
        assert not g.untouched()


SHARED = {
    "one sequence": ([(0, [70])], 1, 4, 4, 128, "f16"),
    "one CTA of the plan": ([(8, [512, 600, 530, 575])], 8, 8, 2, 128, "bf16"),
    "a cluster of the plan": ([(100, [6400 + 31 * i for i in range(40)])], 1, 24, 4, 256, "bf16"),
    "its largest rows": ([(70, [4490 + i for i in range(64)])], 1, 4, 1, 128, "f16"),
    "sequences laid out in memory": ([(3, [192 + i % 70 for i in range(300)])], 2, 2, 1, 128, "bf16"),
    "groups laid out in memory": ([(2, [130, 140, 128 + i % 9]) for i in range(270)], 1, 2, 2, 128, "f16"),
    "pairs": ([(20, [1300, 1400, 1350])], 24, 12, 2, 256, "bf16"),
    "odd heads": ([(9, [600, 610]), (0, [0, 5])], 3, 15, 5, 128, "f16"),
    "a large group": (fork(10, 32, 32), 1, 24, 4, 256, "bf16"),
    "a large group in pairs": (fork(8, 20, 20), 22, 12, 2, 128, "f16"),
    "heads of a whole block": ([(4, [300, 290, 280])], 5, 128, 1, 128, "f16"),
}


@pytest.mark.parametrize("name", list(SHARED))
@pytest.mark.parametrize("out", ["f32", "same"])
def test_plan_and_attention(cuda_dev, name, out):
    LT, case = _lt(), SHARED[name]
    s = make(*case, seed=len(name))
    t = torch.float32 if out == "f32" else s["q"].dtype
    d = {k: v.cuda() for k, v in s.items()}
    (B, N, Hq, D), Hkv, groups = s["q"].shape, s["k_tree"].shape[2], s["group_start"].numel() - 1
    g = Guarded()
    plan = g.take((LT.lucetree_shared_plan_bytes(B, N, Hq, Hkv, D, groups),), torch.uint8)
    ws = g.take((LT.lucetree_verify_attn_shared_workspace(B, N, Hq, Hkv, D, groups),), torch.uint8)
    shared, o, lse = g.take((groups,), torch.int32), g.take((B, N, Hq, D), t), g.take((B, N, Hq), torch.float32)
    inputs = {k: d[k].clone() for k in ("k_pool", "v_pool", "page_table", "ctx_len", "group_start", "q", "anc_mask")}
    status = g.take((1,), torch.int32)
    status.zero_()
    for _ in range(2):
        LT.lucetree_shared_plan(d["page_table"], d["ctx_len"], d["group_start"], N, Hq, Hkv, D, d["k_pool"].shape[0], shared, plan,
                                status)
        LT.lucetree_verify_attn_shared(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"], d["v_tree"],
                                       d["anc_mask"], groups, plan, o, status, ws, lse=lse)
    assert g.untouched() and int(status.item()) == 0
    for k, v in inputs.items():
        assert torch.equal(v.view(torch.uint8), d[k].view(torch.uint8))
    near(o.cpu(), lse.cpu(), reference(s, p_step=P_STEP[t]))


#       B, N, Hq, Hkv, D, rot, layout, dtype
ROPE = [(1, 1, 1, 1, 16, 2, 0, "f16"), (3, 22, 24, 4, 256, 64, 0, "bf16"), (2, 7, 3, 1, 80, 20, 0, "f16"),
        (2, 5, 6, 3, 272, 250, 1, "bf16"), (4, 16, 2, 1, 1024, 1024, 0, "bf16")]


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_rotation(cuda_dev, case):
    LT = _lt()
    B, N, Hq, Hkv, D, rot, layout, dtype = case
    t, g = TYPES[dtype], Guarded()
    q, k, v = (torch.randn(B, N, h, D, device="cuda").to(t) for h in (Hq, Hkv, Hkv))
    outs, status = [g.take(x.shape, t) for x in (q, k, v)], g.take((1,), torch.int32)
    status.zero_()
    steps = LT.lucetree_rope_steps(rot, 10000.0)[0].cuda()
    pos = torch.arange(B * N, dtype=torch.int32, device="cuda").view(B, N)
    LT.lucetree_rope(q, k, steps, layout, outs[0], outs[1], status, positions=pos, v=v, v_out=outs[2])
    assert g.untouched() and int(status.item()) == 0 and torch.equal(outs[2], v)


@pytest.mark.parametrize("case", [(16, "same", "same", "f16", 0), (80, "same", "same", "bf16", 1), (256, "e4m3", "int8", "bf16", 0),
                                  (256, "e4m3", "int4", "bf16", 1), (256, "same", "int4", "f16", 0), (1024, "same", "same", "bf16", 0)],
                         ids=str)
def test_append(cuda_dev, case):
    LT = _lt()
    D, kf, vf, dtype, layout = case
    t, g, Hq, Hkv = TYPES[dtype], Guarded(), 5, 2
    new, ctx = [1, 0, 130, 64, 7], [63, 64, 0, 100, 0]
    B, T, pages = len(new), sum(new), [-(-(n + L) // 64) for n, L in zip(new, ctx)]
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table, at = np.full((B, max(pages)), -1, np.int32), 0
    for b, n in enumerate(pages):  # (the first and the last page of the pool are used)
        table[b, :n] = range(at, at + n)
        at += n
    cuda = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    q, k, v = (torch.randn(T, h, D, device="cuda").to(t) for h in (Hq, Hkv, Hkv))
    kp = g.take((at, Hkv, 64, D), torch.uint8 if kf != "same" else t)
    vp = g.take((at, Hkv, 64, D // 2 if vf == "int4" else D), torch.uint8 if vf != "same" else t)
    exps = [g.take((at, Hkv, 64), torch.uint8) if f != "same" else None for f in (kf, vf)]
    q_out, length, status = g.take((T, Hq, D), t), g.take((B,), torch.int32), g.take((1,), torch.int32)
    status.zero_()
    LT.lucetree_append_kv(k, v, cuda(start), cuda(table), cuda(ctx), length, kp, vp, status, q=q, q_out=q_out,
                          steps=LT.lucetree_rope_steps(D, 10000.0)[0].cuda(), layout=layout, k_exp=exps[0], v_exp=exps[1],
                          v_format={"same": LT.LUCETREE_V_SAME, "int8": LT.LUCETREE_V_INT8, "int4": LT.LUCETREE_V_INT4}[vf])
    assert g.untouched() and int(status.item()) == 0 and length.tolist() == [n + L for n, L in zip(new, ctx)]
    # slots that no row went to are as they were
    written = torch.zeros(at, 64, dtype=torch.bool)
    for b in range(B):
        for p in range(ctx[b], ctx[b] + new[b]):
            written[table[b, p // 64], p % 64] = True
    for buf in (kp, vp, *exps):
        if buf is not None:
            rest = buf.transpose(1, 2)[~written.cuda()].contiguous().view(torch.uint8)
            assert bool((rest == FILL).all())
