// Instantiations of the shared-prefix attention kernel: fp16 operands, head dim 256.
#include "attn_shared_tc.cuh"

namespace lucetree {
namespace shr {

cudaError_t launch_f16_256(const Maps& m, const Launch& W, cudaStream_t stream) {
    return launch_one<256, false, false>(m, W, stream);
}

}  // namespace shr
}  // namespace lucetree
