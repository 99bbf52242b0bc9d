// Instantiations of the tensor-core prefix kernel with a sliding window and sinks, bf16 operands, head
// dim 128; dispatch over the output type.
#include "attn_prefix_tc.cuh"

namespace lucetree {

cudaError_t launch_prefix_tc_bf16_128_win16(int rgp, const CUtensorMap& tk, const CUtensorMap& tv,
                                            const CUtensorMap& tq, const AttnLaunch& L, cudaStream_t stream);

cudaError_t launch_prefix_tc_bf16_128_win(int rgp, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                                          const AttnLaunch& L, cudaStream_t stream) {
    if (L.out_dtype == LUCETREE_BF16) return launch_prefix_tc_bf16_128_win16(rgp, tk, tv, tq, L, stream);
    return prefix_tc::launch_rgp<128, true, 0, 0, 1>(rgp, tk, tv, tq, tv, tv, L, stream);
}

}  // namespace lucetree
