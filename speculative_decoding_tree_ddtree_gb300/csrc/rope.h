// rope.h -- host entry points of the rotary positions and of the appends to the
// paged cache.
#pragma once

#include <cuda_runtime.h>

#include "lucetree.h"

namespace lucetree {

cudaError_t launch_rope(const lucetree_rope_args& a, cudaStream_t stream);
cudaError_t launch_append_kv(const lucetree_append_args& a, cudaStream_t stream);

}  // namespace lucetree
