// attn_merge_win.cu -- the merge launch of lucetree_verify_attn_win: one CTA
// per output row (the routine is in attn_merge.cuh).
#include "attn_merge.cuh"

namespace lucetree {

namespace {

constexpr int kWarps = 4;  // per output row, as in the merge launch of the full attention
constexpr int kThreads = 32 * kWarps;

template <typename T, int D, typename TO>
__global__ void __launch_bounds__(kThreads, 5) merge_win_kernel(AttnLaunch L) {
    __shared__ float s_o[kWarps][D];
    __shared__ float s_red[kWarps];
    if (threadIdx.x == 0) pdl_trigger();
    const long long row = blockIdx.x;
    const int i = (int)((row / L.plan.Hq) % L.plan.N);
    const int b = (int)(row / ((long long)L.plan.Hq * L.plan.N));
    merge::merge_row<T, D, kWarps, 1, true, TO>(L, row, L.a.anc_mask[(size_t)b * L.plan.N + i], s_o, s_red);
}

template <typename T, int D>
cudaError_t launch(const AttnLaunch& L, cudaStream_t stream) {
    const dim3 grid((unsigned)((long long)L.plan.B * L.plan.N * L.plan.Hq)), block(kThreads);
    if (L.out_dtype == LUCETREE_F32) return launch_pdl(merge_win_kernel<T, D, float>, grid, block, 0, stream, L);
    return launch_pdl(merge_win_kernel<T, D, T>, grid, block, 0, stream, L);
}

}  // namespace

cudaError_t launch_attn_merge_win(const AttnLaunch& L, cudaStream_t stream) {
    if (L.a.dtype == LUCETREE_BF16)
        return L.a.D == 256 ? launch<__nv_bfloat16, 256>(L, stream) : launch<__nv_bfloat16, 128>(L, stream);
    return L.a.D == 256 ? launch<__half, 256>(L, stream) : launch<__half, 128>(L, stream);
}

}  // namespace lucetree
