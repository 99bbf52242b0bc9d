// Instantiations of the windowed attention kernel: bf16 operands, head dim 128.
#include "attn_window_tc.cuh"

namespace lucetree {
namespace win {

cudaError_t launch_bf16_128(const Maps& m, const WinLaunch& W, cudaStream_t stream) {
    return launch_rgp<128, true, false>(m, W, stream);
}

}  // namespace win
}  // namespace lucetree
