// Host-side launch interface between the C ABI of the operators around the finalize (layer_api.cu) and
// their kernels, and the launch helper they share.
#pragma once

#include <cuda_runtime.h>

#include "mfr_device.cuh"
#include "moe_layer.h"

namespace mfr {

// The tokens of a batch are cut into at most kRouteBlocks contiguous chunks, one CTA each.  One per SM of a
// GB300; a constant, so that the workspace does not depend on the device.
constexpr int kRouteBlocks = 152;
// Batches of at most this many tokens are routed and ordered by one CTA in one launch, with no workspace.
constexpr int kRouteOneBlockTokens = 64;
// CTAs of the head-norm gradient at most: two on each SM of a GB300, a row of partial weight gradients each.
constexpr int kHeadGradBlocks = 152 * 2;

inline int route_blocks(int T) {
  if (T <= kRouteOneBlockTokens) return 1;
  return T < kRouteBlocks ? T : kRouteBlocks;
}

cudaError_t launch_route(const mfr_route_args& a, cudaStream_t stream);
cudaError_t launch_route_backward(const mfr_route_backward_args& a, cudaStream_t stream);
cudaError_t launch_dispatch(const mfr_dispatch_args& a, cudaStream_t stream);
cudaError_t launch_routed_backward(const mfr_routed_backward_args& a, cudaStream_t stream);
// Rows of partial weight gradients ([2][D] FP32 each) that the head-norm gradient leaves in its workspace.
int head_grad_rows(int T, int q_heads, int k_heads, int D);
cudaError_t launch_head_norm(const mfr_head_norm_args& a, cudaStream_t stream);
cudaError_t launch_head_norm_backward(const mfr_head_norm_args& a, cudaStream_t stream);

// Launch `kern` with the programmatic-dependent-launch attribute iff `pdl`.  Every kernel launched this way
// waits (pdl_wait) before it reads or writes anything.
template <typename P>
cudaError_t launch_pdl(void (*kern)(const P), dim3 grid, int block, int smem, bool pdl, cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace mfr
