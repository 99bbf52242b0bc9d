// pages.h -- host entry points of the page-table operations and of the page and
// state copies that go with them.
#pragma once

#include <cuda_runtime.h>

#include "lucetree.h"

namespace lucetree {

size_t reorder_workspace_bytes(int rows_in, int rows_out, int num_pages);
cudaError_t launch_reorder_pages(const lucetree_reorder_args& a, void* workspace, cudaStream_t stream);
cudaError_t launch_trim_pages(const lucetree_trim_args& a, cudaStream_t stream);
size_t compact_workspace_bytes(int num_pages);
cudaError_t launch_compact_pages(const lucetree_compact_args& a, void* workspace, cudaStream_t stream);
cudaError_t launch_copy_pages(const lucetree_copy_pages_args& a, cudaStream_t stream);
cudaError_t launch_reorder_states(const lucetree_reorder_states_args& a, cudaStream_t stream);

}  // namespace lucetree
