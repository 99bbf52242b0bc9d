"""The full attention, its forms over quantised K and V and the fused step, with scores that
rise steeply from one key tile to the next."""
import pytest
import torch

from tests.test_gpu_attention_steep import compare, raise_keys
from tests.test_gpu_attention_window import make

pytestmark = pytest.mark.gpu

SHAPES = {
    "128":  ((1000, 700, 930, 64, 0) * 9, 3, 8, 4, 128),
    "256":  ((900, 500) * 14, 3, 12, 4, 256),
    "wide": ((700,) * 13, 22, 24, 4, 256),
}
RAISE = {"one": ([351, 620], [95.0, 300.0]), "stairs": (range(140, 1000, 70), [100.0 * k for k in range(1, 14)])}


def _lt():
    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    return LT


def inputs(shape, dtype):
    ctx, N, Hq, Hkv, D = SHAPES[shape]
    return make(ctx, N, Hq, Hkv, D, dtype, 1 << 20, 0, "chain", seed=33)


def run(s, entry, workspace, *args, names=("q", "k_pool", "v_pool"), scale=None, **kw):
    B, N, Hq, D = s["q"].shape
    d = {k: v.cuda() for k, v in s.items() if torch.is_tensor(v)}
    out = torch.full((B, N, Hq, D), float("nan"), device="cuda")
    lse = torch.full((B, N, Hq), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(workspace(B, N, Hq, s["k_tree"].shape[2], D), dtype=torch.uint8, device="cuda")
    entry(*(d[n] for n in names), *args, d["page_table"], d["ctx_len"], d["k_tree"], d["v_tree"], d["anc_mask"], out, st, ws,
          lse=lse, scale=scale, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), int(st.item())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("how", ["scale", "one", "stairs"])
def test_full(cuda_dev, shape, dtype, how):
    LT = _lt()
    s, scale = inputs(shape, dtype), 20.0 if how == "scale" else None
    if how != "scale":
        raise_keys(s, *RAISE[how])
    compare(s, *run(s, LT.lucetree_verify_attn, LT.lucetree_verify_attn_workspace, scale=scale), torch.float32, scale)


@pytest.mark.parametrize("shape", ["256", "wide"])
def test_quantised_v(cuda_dev, shape):
    # codes of 8 bits at 2^-5: the values are bf16 numbers, so the formula sees what the kernel sees
    LT = _lt()
    s = raise_keys(inputs(shape, "bf16"), *RAISE["one"])
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(-127, 128, s["v_pool"].shape, generator=g, dtype=torch.int8)
    s["v_pool"] = (codes.float() / 32).bfloat16()
    s["v_codes"], s["v_exp"] = codes, torch.full(codes.shape[:3], 122, dtype=torch.uint8)
    got = run(s, LT.lucetree_verify_attn_vq, LT.lucetree_verify_attn_workspace, LT.LUCETREE_V_INT8,
              names=("q", "k_pool", "v_codes", "v_exp"))
    compare(s, *got, torch.float32)


@pytest.mark.parametrize("shape", ["256", "wide"])
def test_quantised_k(cuda_dev, shape):
    # queries of 1/2 are exact in the kernel's two parts; E4M3 values are bf16 numbers
    LT = _lt()
    s = inputs(shape, "bf16")
    g = torch.Generator().manual_seed(2)
    codes = torch.randint(0, 0x30, s["k_pool"].shape, generator=g, dtype=torch.uint8)  # up to 1/2
    codes |= (torch.rand(codes.shape, generator=g) < 0.5).to(torch.uint8) << 7
    exps = torch.full(codes.shape[:3], 127, dtype=torch.uint8)
    s["q"] = torch.full_like(s["q"], 0.5)
    for b, L in enumerate(s["ctx_len"].tolist()):
        for p, e in ((351, 131), (620, 133)):        # 1 x 2^4 and 2^6: 128 and 512 nats
            if p < L:
                page = int(s["page_table"][b, p // 64])
                codes[page, :, p % 64], exps[page, :, p % 64] = 0x38, e
    values = codes.view(torch.float8_e4m3fn).float() * torch.exp2(exps.float() - 127)[..., None]
    s["k_pool"], s["k_codes"], s["k_exp"] = values.bfloat16(), codes, exps
    got = run(s, LT.lucetree_verify_attn_kq, LT.lucetree_verify_attn_kq_workspace, names=("q", "k_codes", "k_exp", "v_pool"))
    compare(s, *got, torch.float32)


def test_fused_step(cuda_dev):
    LT = _lt()
    s = raise_keys(inputs("128", "bf16"), *RAISE["stairs"])
    B, N, Hq, D = s["q"].shape
    d = {k: v.cuda() for k, v in s.items() if torch.is_tensor(v)}
    vocab = 64
    parent = torch.arange(-1, N - 1, dtype=torch.int32).expand(B, N).contiguous().cuda()
    draft = torch.zeros(B, N, dtype=torch.int32, device="cuda")
    logits = torch.zeros(B, N + 1, vocab, device="cuda")
    logits[..., 5] = 1.0                             # no draft is accepted: the pool stays as it is
    step = LT.VerifyStep(B, N, Hq, 4, D, vocab)
    step.run(d["q"], d["k_pool"], d["v_pool"], d["page_table"], d["ctx_len"], d["k_tree"], d["v_tree"], parent, draft, logits)
    torch.cuda.synchronize()
    assert (step.acc_len == 0).all()
    compare(s, step.out.cpu(), step.lse.cpu(), int(step.status.item()), torch.float32)
