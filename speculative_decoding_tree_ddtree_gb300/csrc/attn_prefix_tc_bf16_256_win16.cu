// Instantiations of the tensor-core prefix kernel with a sliding window and sinks, bf16 operands and a
// bf16 output, head dim 256.
#include "attn_prefix_tc.cuh"

namespace lucetree {

cudaError_t launch_prefix_tc_bf16_256_win16(int rgp, const CUtensorMap& tk, const CUtensorMap& tv,
                                            const CUtensorMap& tq, const AttnLaunch& L, cudaStream_t stream) {
    return prefix_tc::launch_rgp<256, true, 0, 0, 2>(rgp, tk, tv, tq, tv, tv, L, stream);
}

}  // namespace lucetree
