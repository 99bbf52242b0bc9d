// attn_merge_win.cu -- the merge launch of lucetree_verify_attn_win (the routine
// is in attn_merge.cuh).
#include "attn_merge.cuh"

namespace lucetree {

namespace {

constexpr int kWarps = 4;  // of a CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 5;

// W warps to a row.  Four (one CTA a row, as in the merge launch of the full
// attention) give the shortest way through one row; with many rows, one warp a row
// keeps four times as many rows in flight.
template <typename T, int D, typename TO, int W>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) merge_win_kernel(AttnLaunch L) {
    __shared__ float s_o[W][D];
    __shared__ float s_red[W];
    if (threadIdx.x == 0) pdl_trigger();
    const int group = W == 1 ? threadIdx.x >> 5 : 0;
    const long long row = (long long)blockIdx.x * (kWarps / W) + group;
    if (row >= (long long)L.plan.B * L.plan.N * L.plan.Hq) return;  // a whole warp, and only with W = 1
    const int i = (int)((row / L.plan.Hq) % L.plan.N);
    const int b = (int)(row / ((long long)L.plan.Hq * L.plan.N));
    merge::merge_row<T, D, W, 1, true, TO>(L, row, L.a.anc_mask[(size_t)b * L.plan.N + i], s_o, s_red, group);
}

template <typename T, int D, typename TO>
cudaError_t launch_out(const AttnLaunch& L, cudaStream_t stream) {
    const long long rows = (long long)L.plan.B * L.plan.N * L.plan.Hq;
    int dev = 0;
    cudaGetDevice(&dev);
    if (rows > 2ll * kCtasPerSm * device_sm_count(dev))
        return launch_pdl(merge_win_kernel<T, D, TO, 1>, dim3((unsigned)((rows + kWarps - 1) / kWarps)), dim3(kThreads), 0,
                          stream, L);
    return launch_pdl(merge_win_kernel<T, D, TO, kWarps>, dim3((unsigned)rows), dim3(kThreads), 0, stream, L);
}

template <typename T, int D>
cudaError_t launch(const AttnLaunch& L, cudaStream_t stream) {
    return L.out_dtype == LUCETREE_F32 ? launch_out<T, D, float>(L, stream) : launch_out<T, D, T>(L, stream);
}

}  // namespace

cudaError_t launch_attn_merge_win(const AttnLaunch& L, cudaStream_t stream) {
    if (L.a.dtype == LUCETREE_BF16)
        return L.a.D == 256 ? launch<__nv_bfloat16, 256>(L, stream) : launch<__nv_bfloat16, 128>(L, stream);
    return L.a.D == 256 ? launch<__half, 256>(L, stream) : launch<__half, 128>(L, stream);
}

}  // namespace lucetree
