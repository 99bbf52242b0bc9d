// Instantiations of the shared-prefix attention kernel: bf16 operands, head dim 128.
#include "attn_shared_tc.cuh"

namespace lucetree {
namespace shr {

cudaError_t launch_bf16_128(const Maps& m, const Launch& W, cudaStream_t stream) {
    return launch_one<128, true, false>(m, W, stream);
}

}  // namespace shr
}  // namespace lucetree
