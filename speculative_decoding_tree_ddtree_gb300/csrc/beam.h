// beam.h -- host entry points of the beam selection.
#pragma once

#include <cuda_runtime.h>

#include "lucetree.h"

namespace lucetree {

size_t beam_workspace_bytes(int batch, int beams, int vocab, int device);
cudaError_t launch_beam_select(const lucetree_beam_args& a, void* workspace, int device, cudaStream_t stream);

}  // namespace lucetree
