// attn_window.cu -- lucetree_verify_attn_win: tree-verify attention in which a
// node sees the last `window` positions up to its own and the first `sinks`
// positions of its sequence.  Argument checks, TMA tensor maps and the two
// launches (attn_window_tc.cuh, attn_window_merge.cu).
#include <cuda.h>

#include "attn_window_tc.cuh"

namespace lucetree {

lucetree_status verify_attn_check(const lucetree_attn_args* a, bool need_mask, int v_format, AttnLaunch* L);

namespace win {

namespace {

cudaError_t launch_window(const WinLaunch& W, cudaStream_t stream) {
    const lucetree_attn_args& a = W.L.a;
    const PlanDims& p = W.L.plan;
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const CUtensorMapDataType dt =
        a.dtype == LUCETREE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint32_t ones[3] = {1, 1, 1};
    auto map = [&](CUtensorMap* m, int rank, const void* at, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
        return enc(m, dt, rank, const_cast<void*>(at), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t D = a.D, row = D * 2;
    Maps m;
    // pools as [num_pages * Hkv * 64 rows][D]; box = one 64-token page x 64 dims
    const cuuint64_t pool_dims[2] = {D, (cuuint64_t)a.num_pages * a.Hkv * kPage}, pool_strides[1] = {row};
    const cuuint32_t pool_box[2] = {64, (cuuint32_t)kPage};
    // queries as [B*N nodes][Hq heads][D]; box = 64 dims x G heads x NPG nodes
    const cuuint64_t q_dims[3] = {D, (cuuint64_t)a.Hq, (cuuint64_t)a.B * a.N}, q_strides[2] = {row, (cuuint64_t)a.Hq * row};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.rg.NPG};
    // tree K/V as [B*N nodes][Hkv][D]; box = 64 dims of one head of a sequence's N nodes
    const cuuint64_t t_dims[3] = {D, (cuuint64_t)a.Hkv, (cuuint64_t)a.B * a.N}, t_strides[2] = {row, (cuuint64_t)a.Hkv * row};
    const cuuint32_t t_box[3] = {64, 1, (cuuint32_t)a.N};
    if (!map(&m.k, 2, a.k_pool, pool_dims, pool_strides, pool_box) || !map(&m.v, 2, a.v_pool, pool_dims, pool_strides, pool_box) ||
        !map(&m.q, 3, a.q, q_dims, q_strides, q_box) || !map(&m.kt, 3, a.k_tree, t_dims, t_strides, t_box) ||
        !map(&m.vt, 3, a.v_tree, t_dims, t_strides, t_box))
        return cudaErrorInvalidValue;
    if (a.dtype == LUCETREE_F16) return a.D == 256 ? launch_f16_256(m, W, stream) : launch_f16_128(m, W, stream);
    if (W.out_dtype == LUCETREE_BF16)
        return a.D == 256 ? launch_bf16_256_out16(m, W, stream) : launch_bf16_128_out16(m, W, stream);
    return a.D == 256 ? launch_bf16_256(m, W, stream) : launch_bf16_128(m, W, stream);
}

// A CTA to each segment where that costs no tile more than an even cut, or one tile where
// that is worth it: it saves the partial sums and the launch that joins them, whose time
// grows with the number of segments, against a tile's, which grows with D and the rows.
// Segment by segment against cut, us, two tiles against one (window 60):
//   D = 128, 4 segments    32 rows  9.1 / 10.2   64  11.1 / 11.3   96  12.4 / 12.5   112  15.5 / 14.5
//            16            32       9.2 / 11.2   64  11.2 / 12.4   96  12.6 / 12.8   112  15.7 / 14.6
//            24            32       9.3 / 10.5   64  11.2 / 11.6   96  12.6 / 13.6   112  15.7 / 16.3
//   D = 256, 4              6      11.7 / 10.7   72  15.2 / 13.6                     132  20.5 / 17.6
//            24             6      11.8 / 11.6   72  15.3 / 14.4                     132  20.5 / 19.4
//            40             6      12.0 / 12.6   72  15.5 / 16.1                     132  20.5 / 21.1
//            60             6      12.1 / 12.8   72  15.7 / 16.9                     132  20.6 / 23.1
// (one tile either way: 30 x 4 segments of 132 rows, D = 256, 18.9 / 21.3)
bool stay_whole(const WinLaunch& W) {
    const PlanDims& p = W.L.plan;
    const long long ctas = (long long)p.S * p.rg.NG;
    if (ctas > grid_ctas(p)) return false;
    const long long most = most_tiles(W.window, W.sinks, p.max_pages), cut = (p.S * most + p.Cg - 1) / p.Cg;
    const bool one_more = p.D == 128 ? p.rg.RG <= 96 || ctas >= 24 : ctas >= 40;
    return most - cut <= (one_more ? 1 : 0);
}

}  // namespace

}  // namespace win
}  // namespace lucetree

using namespace lucetree;

extern "C" lucetree_status lucetree_verify_attn_win(const lucetree_win_args* w, void* workspace,
                                                    size_t workspace_bytes, void* stream) {
    if (!w) return LUCETREE_ERR_INVALID_ARG;
    if (w->window < 1 || w->sinks < 0 || !w->out) return LUCETREE_ERR_INVALID_ARG;
    if (w->out_dtype != LUCETREE_F32 && w->out_dtype != w->attn.dtype) return LUCETREE_ERR_UNSUPPORTED;
    lucetree_attn_args a = w->attn;
    a.out = reinterpret_cast<float*>(w->out);  // checked like the full attention's; written as out_dtype
    win::WinLaunch W;
    const lucetree_status st = verify_attn_check(&a, true, LUCETREE_V_SAME, &W.L);
    if (st != LUCETREE_OK) return st;
    // 32-bit row and flat tile numbers (a segment has at most one tile more than its prefix: the tree's page)
    const long long tiles = ((long long)a.max_pages_per_seq + 2) / 2;
    if ((long long)a.B * a.N * a.Hq > 0x7fffffffll || (long long)a.B * a.Hkv * tiles > 0x7fffffffll)
        return LUCETREE_ERR_UNSUPPORTED;
    // rows are written while others are still to be read
    const long long rows = (long long)a.B * a.N, q_elems = rows * a.Hq * a.D, t_bytes = rows * a.Hkv * a.D * 2;
    const long long out_bytes = q_elems * (w->out_dtype == LUCETREE_F32 ? 4 : 2);
    if (bytes_overlap(w->out, out_bytes, a.q, q_elems * 2) || bytes_overlap(w->out, out_bytes, a.k_tree, t_bytes) ||
        bytes_overlap(w->out, out_bytes, a.v_tree, t_bytes))
        return LUCETREE_ERR_INVALID_ARG;
    W.window = w->window;
    W.sinks = w->sinks;
    W.out_dtype = w->out_dtype;
    W.out = w->out;
    if (!workspace || workspace_bytes < attn_workspace_bytes(W.L.plan) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return LUCETREE_ERR_WORKSPACE;
    W.L.ws = reinterpret_cast<float*>(workspace);
    W.alone = win::stay_whole(W);
    if (W.alone) W.L.plan.Cg = W.L.plan.S;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (win::launch_window(W, s) != cudaSuccess) return LUCETREE_ERR_CUDA;
    if (!W.alone && win::launch_merge(W, s) != cudaSuccess) return LUCETREE_ERR_CUDA;
    return LUCETREE_OK;
}
