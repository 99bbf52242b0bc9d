// Instantiations of the tensor-core prefix kernel with a sliding window and sinks, f16 operands, head
// dim 256; dispatch over the head dim.
#include "attn_prefix_tc.cuh"

namespace lucetree {

cudaError_t launch_prefix_tc_f16_128_win(int rgp, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                                          const AttnLaunch& L, cudaStream_t stream);

cudaError_t launch_prefix_tc_f16_win(int rgp, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                                      const AttnLaunch& L, cudaStream_t stream) {
    if (L.a.D == 128) return launch_prefix_tc_f16_128_win(rgp, tk, tv, tq, L, stream);
    return prefix_tc::launch_rgp<256, false, 0, 0, 1>(rgp, tk, tv, tq, tv, tv, L, stream);
}

}  // namespace lucetree
