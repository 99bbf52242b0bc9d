// Instantiations of the shared-prefix attention kernel: bf16 operands, head dim 256, 16-bit output with P in bf16.
#include "attn_shared_tc.cuh"

namespace lucetree {
namespace shr {

cudaError_t launch_bf16_256_out16(const Maps& m, const Launch& W, cudaStream_t stream) {
    return launch_one<256, true, true>(m, W, stream);
}

}  // namespace shr
}  // namespace lucetree
