// Instantiations of the windowed attention kernel: bf16 operands, head dim 256, 16-bit output with P in bf16.
#include "attn_window_tc.cuh"

namespace lucetree {
namespace win {

cudaError_t launch_bf16_256_out16(const Maps& m, const WinLaunch& W, cudaStream_t stream) {
    return launch_rgp<256, true, true>(m, W, stream);
}

}  // namespace win
}  // namespace lucetree
