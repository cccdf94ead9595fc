// Host-side launch interface between the C ABI of the operators around the finalize (layer_api.cu) and
// their kernels, and the launch helper they share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "mfr_device.cuh"
#include "moe_layer.h"

namespace mfr {

// The tokens of a batch are cut into at most kRouteBlocks contiguous chunks, one CTA each.  One per SM of a
// GB300; a constant, so that the workspace does not depend on the device.
constexpr int kRouteBlocks = 152;
// With the expert order a chunk has at least so many tokens as one SM routes about as fast as one (the instructions of
// a token grow with the experts that a lane holds), since the order reads every chunk's counts in every CTA; and
// batches of at most kRouteCluster chunks (the portable cluster size) run as one cluster, in one launch and with no
// workspace.  Measured on GB300, in a graph: 128 tokens of 256 experts (top-8) 5.4 us in a cluster of 8, 5.9 in one of 4;
// 256 tokens 6.1 in two launches, 6.2 in a cluster of 8; 128 tokens of 896 experts (top-16) 9.8, and 15.5 with a chunk
// for each token.
constexpr int kRouteCluster = 8;
inline int route_cta_tokens(int E) { return E <= 256 ? 16 : E <= 512 ? 8 : 4; }

// CTAs of the head-norm gradient at most: two on each SM of a GB300, a row of partial weight gradients each.
constexpr int kHeadGradBlocks = 152 * 2;

inline int route_chunks(int T, int E, bool order) {
  if (T == 0) return 1;
  const int per = route_cta_tokens(E);
  // (the order reads every chunk's counts in every CTA: no more chunks than the routing gains from)
  const int want = order ? (T + per - 1) / per : T;
  return want < kRouteBlocks ? want : kRouteBlocks;
}

cudaError_t launch_route(const mfr_route_args& a, cudaStream_t stream);
cudaError_t launch_route_backward(const mfr_route_backward_args& a, cudaStream_t stream);
cudaError_t launch_dispatch(const mfr_dispatch_args& a, cudaStream_t stream);
cudaError_t launch_routed_backward(const mfr_routed_backward_args& a, cudaStream_t stream);
// Rows of partial weight gradients ([2][D] FP32 each) that the head-norm gradient leaves in its workspace.
int head_grad_rows(int T, int q_heads, int k_heads, int D);
cudaError_t launch_head_norm(const mfr_head_norm_args& a, cudaStream_t stream);
cudaError_t launch_head_norm_backward(const mfr_head_norm_args& a, cudaStream_t stream);

// Lets Kern have up to `most` bytes of dynamic shared memory on the current device: once a device, since the runtime's
// call costs as much as a small launch's preparation.
template <auto Kern>
cudaError_t allow_smem(int most) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch `kern` in clusters of `cluster` CTAs, with the programmatic-dependent-launch attribute iff `pdl`.  Every kernel
// launched this way waits (pdl_wait) before it reads or writes anything.
template <typename P>
cudaError_t launch_pdl(void (*kern)(const P), dim3 grid, int block, int smem, bool pdl, cudaStream_t stream, const P& p, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace mfr
