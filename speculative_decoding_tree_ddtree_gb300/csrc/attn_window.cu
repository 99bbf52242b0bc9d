// attn_window.cu -- lucetree_verify_attn_win: tree-verify attention in which a
// node sees the last `window` positions up to its own and the first `sinks`
// positions of its sequence.  The kernels are those of the full attention,
// compiled for the window's key list (prefix_tc_kernel<.., WIN>, merge_row
// with WIN).
#include "internal.cuh"

namespace lucetree {
lucetree_status verify_attn_check(const lucetree_attn_args* a, bool need_mask, int v_format, AttnLaunch* L);
}

using namespace lucetree;

extern "C" lucetree_status lucetree_verify_attn_win(const lucetree_win_args* w, void* workspace,
                                                    size_t workspace_bytes, void* stream) {
    if (!w) return LUCETREE_ERR_INVALID_ARG;
    if (w->window < 1 || w->sinks < 0 || !w->out) return LUCETREE_ERR_INVALID_ARG;
    if (w->out_dtype != LUCETREE_F32 && w->out_dtype != w->attn.dtype) return LUCETREE_ERR_UNSUPPORTED;
    lucetree_attn_args a = w->attn;
    a.out = reinterpret_cast<float*>(w->out);  // written as out_dtype
    AttnLaunch L;
    const lucetree_status st = verify_attn_check(&a, true, LUCETREE_V_SAME, &L);
    if (st != LUCETREE_OK) return st;
    if ((long long)a.B * a.N * a.Hq > 0x7fffffffll) return LUCETREE_ERR_UNSUPPORTED;  // one merge CTA per row
    L.plan.window = w->window;
    L.plan.sinks = w->sinks;
    L.out_dtype = w->out_dtype;
    if (!workspace || workspace_bytes < attn_workspace_bytes(L.plan) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return LUCETREE_ERR_WORKSPACE;
    L.ws = reinterpret_cast<float*>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (launch_attn_prefix(L, s) != cudaSuccess) return LUCETREE_ERR_CUDA;
    if (launch_attn_merge_win(L, s) != cudaSuccess) return LUCETREE_ERR_CUDA;
    return LUCETREE_OK;
}
