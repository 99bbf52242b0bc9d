"""Shared-prefix plan and attention at their edges: calls that follow each other closely."""
import pytest
import torch

from tests.shared_cases import PAGE, TYPES
from tests.test_gpu_attention_shared import P_STEP, _lt, make, near, reference

pytestmark = pytest.mark.gpu


class Call:
    """A plan and an attention call with buffers of their own, for repeated calls."""

    def __init__(self, s, out_dtype=torch.float32, start=None):
        LT = _lt()
        self.d = {k: v.cuda() for k, v in s.items()}
        if start is not None:
            self.d["group_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        (B, N, Hq, D), Hkv, groups = s["q"].shape, s["k_tree"].shape[2], self.d["group_start"].numel() - 1
        self.N, self.Hq, self.Hkv, self.D, self.groups = N, Hq, Hkv, D, groups
        self.out = torch.full((B, N, Hq, D), float("nan"), dtype=out_dtype, device="cuda")
        self.lse = torch.full((B, N, Hq), float("nan"), device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.shared = torch.empty(groups, dtype=torch.int32, device="cuda")
        self.plan = torch.empty(LT.lucetree_shared_plan_bytes(B, N, Hq, Hkv, D, groups), dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(LT.lucetree_verify_attn_shared_workspace(B, N, Hq, Hkv, D, groups), dtype=torch.uint8, device="cuda")
        self.ws.fill_(0x7F)

    def make_plan(self):
        d = self.d
        _lt().lucetree_shared_plan(d["page_table"], d["ctx_len"], d["group_start"], self.N, self.Hq, self.Hkv, self.D,
                                   d["k_pool"].shape[0], self.shared, self.plan, self.status)

    def attend(self):
        d = self.d
        _lt().lucetree_verify_attn_shared(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"], d["v_tree"],
                                          d["anc_mask"], self.groups, self.plan, self.out, self.status, self.ws, lse=self.lse)

    def run(self):
        self.make_plan()
        self.attend()
        torch.cuda.synchronize()
        return self.out.cpu(), self.lse.cpu(), int(self.status.item())


# (in pairs of CTAs: a tile or two to a pair, and segments that several pairs share; one CTA to a block)
CLOSE = [
    ([(1, [70, 80, 90])], 22, 12, 2, 256, "bf16"), ([(40, [2600, 2700, 2650, 2601])], 12, 24, 4, 128, "f16"),
    ([(0, [0, 0, 0])], 16, 8, 2, 128, "f16"), ([(8, [512, 600])], 1, 8, 2, 256, "bf16"),
]


def test_calls_that_follow_each_other_closely(cuda_dev):
    """CTAs take over shared and tensor memory from CTAs of other calls that have just left, hundreds of times: with
    barriers in other places, in other phases."""
    calls = [Call(make(*c, seed=30 + i), t) for i, c in enumerate(CLOSE) for t in (torch.float32, TYPES[c[5]])]
    first = [c.run() for c in calls]
    for _ in range(60):
        for c in calls:
            c.out.fill_(float("nan"))
        for c in calls:
            c.attend()
        for c in reversed(calls):
            c.attend()
    torch.cuda.synchronize()
    for c, (out, lse, status) in zip(calls, first):
        assert status == 0 == int(c.status.item())
        assert torch.equal(c.out.cpu(), out) and torch.equal(c.lse.cpu(), lse)


def test_closely_following_calls_match_the_formula(cuda_dev):
    for i, c in enumerate(CLOSE):
        s = make(*c, seed=30 + i)
        out, lse, status = Call(s).run()
        assert status == 0
        near(out, lse, reference(s, p_step=P_STEP[torch.float32]))


BROKEN = [([(10, [700, 650, 800, 641])], 3, 8, 2, 128, "bf16"), ([(10, [700, 650, 641, 720])], 12, 8, 2, 256, "bf16"),
          ([(10, [3700, 650, 641, 720])], 2, 6, 2, 128, "f16"), ([(200, [13000, 12900, 12950, 12800])], 1, 24, 4, 256, "bf16")]


@pytest.mark.parametrize("case", BROKEN, ids=str)
@pytest.mark.parametrize("out", ["f32", "same"])
def test_values_that_are_not_finite_whatever_the_groups(cuda_dev, case, out):
    """One committed V in a sequence's own page, or in a common one: all dims and the lse of the rows that see it are
    NaN, and the others' within their bounds, with the batch as one group, as groups of one, and in between."""
    LT = _lt()
    s = make(*case, seed=41)
    B, N, Hq, D = s["q"].shape
    G, t = Hq // s["k_tree"].shape[2], torch.float32 if out == "f32" else s["q"].dtype
    ref = reference(s, p_step=P_STEP[t])
    values = [float("nan"), float("-inf")] + ([65536.0] if case[5] == "bf16" and t == torch.float32 else [])
    places = [(1, int(s["ctx_len"][1]) - 1, 0), (B - 1, 64, D - 1)]  # own, common
    for start in ([0, B], list(range(B + 1)), [0, 2, B], [0, 1, B], [0, B - 1, B]):
        for b, pos, dim in places:
            for value in values:
                x = dict(s, v_pool=s["v_pool"].clone())
                page = int(s["page_table"][b, pos // PAGE])
                x["v_pool"][page, 1, pos % PAGE, dim] = value
                got, lse, status = Call(x, t, start).run()
                assert status == LT.DEV_NONFINITE
                good = torch.ones(B, N, Hq, dtype=torch.bool)
                seen = torch.tensor([page in s["page_table"][c, :-(-int(s["ctx_len"][c]) // PAGE)].tolist() for c in range(B)])
                good[seen, :, G:2 * G] = False
                near(got, lse, ref, good)
                assert bool(torch.isnan(got[~good]).all()) and bool(torch.isnan(lse[~good]).all())
