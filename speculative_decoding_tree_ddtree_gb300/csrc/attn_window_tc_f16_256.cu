// Instantiations of the windowed attention kernel: f16 operands, head dim 256.
#include "attn_window_tc.cuh"

namespace lucetree {
namespace win {

cudaError_t launch_f16_256(const Maps& m, const WinLaunch& W, cudaStream_t stream) {
    return launch_rgp<256, false, false>(m, W, stream);
}

}  // namespace win
}  // namespace lucetree
