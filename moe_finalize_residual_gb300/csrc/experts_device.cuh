// What the experts' products share: bounded waits, the expert's rows on the device, tensor maps, zeroing of the rows of
// no expert.
#pragma once

#include <cudaTypedefs.h>

#include "experts_launch.h"
#include "mma_device.cuh"

namespace mfr {

constexpr uint64_t kExpertWaitNs = 2000000000ull;

// Bounded wait on an mbarrier phase: false if the CTA is giving up or the limit (about 2 s) ran out; that is counted, and
// starts the giving up.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* give_up, unsigned int* timeouts) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 15u) == 0) {
      if (*give_up) return false;
      if (global_timer_ns() - t0 > kExpertWaitNs) {
        atomicAdd(timeouts, 1u);
        *give_up = 1;
        return false;
      }
    }
  }
}

// The rows of expert e, cut to [0, R]: whatever the device data says, no row outside is touched.
struct RowSpan {
  int begin, end;
};
__device__ __forceinline__ RowSpan expert_rows(const int32_t* offsets, const int32_t* counts, int e, int R) {
  const int64_t b = offsets[e];
  const int64_t n = counts != nullptr ? static_cast<int64_t>(counts[e]) : static_cast<int64_t>(offsets[e + 1]) - b;
  RowSpan s;
  s.begin = static_cast<int>(b < 0 ? 0 : b > R ? R : b);
  const int64_t end = b + n;
  s.end = static_cast<int>(end < s.begin ? s.begin : end > R ? R : end);
  return s;
}

// first[e] = the tiles of `tile` rows of the experts before e, e = 0..E, by all threads of the CTA; `scratch` holds 33 ints.
__device__ __forceinline__ void count_tiles(int* first, int* scratch, const int32_t* offsets, const int32_t* counts, int E, int R, int tile) {
  const int n = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int per = (E + n - 1) / n;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int e = t * per + i;
    if (e < E) {
      const RowSpan s = expert_rows(offsets, counts, e, R);
      sum += (s.end - s.begin + tile - 1) / tile;
    }
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) scratch[warp] = before;
  __syncthreads();
  int at = before - sum;
  for (int w = 0; w < warp; ++w) at += scratch[w];
  for (int i = 0; i < per; ++i) {
    const int e = t * per + i;
    if (e < E) {
      const RowSpan s = expert_rows(offsets, counts, e, R);
      first[e] = at;
      at += (s.end - s.begin + tile - 1) / tile;
    }
  }
  if (t == n - 1) first[E] = at;
  __syncthreads();
}

// The expert of tile number m < first[E].
__device__ __forceinline__ int tile_expert(const int* first, int E, int m) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= m) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Zeros in the rows of no expert of an output with `bytes` (a multiple of 16) a row, by `nwarps` warps (this one is `w`).
// Gap g lies behind the rows of expert g - 1; a warp looks at 32 gaps at a time.
__device__ __forceinline__ void zero_free_rows(uint8_t* out, int64_t stride_bytes, int64_t bytes, const int32_t* offsets,
                                               const int32_t* counts, int E, int R, int w, int nwarps) {
  const int lane = threadIdx.x & 31;
  for (int g0 = 0; g0 <= E; g0 += 32) {
    const int g = g0 + lane;
    int begin = 0, end = 0;
    if (g <= E) {
      begin = g > 0 ? expert_rows(offsets, counts, g - 1, R).end : 0;
      end = g < E ? expert_rows(offsets, counts, g, R).begin : R;
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, end > begin); left != 0; left &= left - 1) {
      const int l = __ffs(left) - 1;
      const int from = __shfl_sync(0xffffffffu, begin, l), to = __shfl_sync(0xffffffffu, end, l);
      // (neighbouring gaps start at neighbouring warps)
      for (int64_t r = from + (w + nwarps - (g0 + l) % nwarps) % nwarps; r < to; r += nwarps)
        for (int64_t i = lane * 16; i < bytes; i += 512) *reinterpret_cast<uint4*>(out + r * stride_bytes + i) = make_uint4(0, 0, 0, 0);
    }
  }
}

// g / (1 + exp(-g)) * u; where exp(-g) is infinite the quotient is 0.
__device__ __forceinline__ float swiglu(float g, float u) { return g * __frcp_rn(1.0f + __expf(-g)) * u; }

// ------------------------------------------------------------------------------------------------
// Tensor maps (host)
// ------------------------------------------------------------------------------------------------

// The driver's encoder, found once.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
        st != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return f;
}

// A map of `rank` dimensions (the first one's values next to one another, `strides` in bytes those of the others) with boxes
// of `box` values, the first 128 bytes, in the 128-byte swizzle; what lies outside reads as zeros.
inline cudaError_t encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* data, int rank, const cuuint64_t* dims,
                              const cuuint64_t* strides, const cuuint32_t* box) {
  const auto f = tensor_map_encoder();
  if (f == nullptr) return cudaErrorNotSupported;
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  const CUresult r = f(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(data), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// Rows: `nx` values, `ny` rows `sy` bytes apart.
inline cudaError_t encode_rows(CUtensorMap* map, CUtensorMapDataType type, const void* data, int64_t nx, int64_t ny, int64_t sy, int bx, int by) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(nx), static_cast<cuuint64_t>(ny)}, strides[1] = {static_cast<cuuint64_t>(sy)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(bx), static_cast<cuuint32_t>(by)};
  return encode_map(map, type, data, 2, dims, strides, box);
}
// Weights: `nz` experts of `ny` rows of `nx` values.
inline cudaError_t encode_weights(CUtensorMap* map, CUtensorMapDataType type, const void* data, int64_t nx, int64_t ny, int64_t nz, int64_t sy,
                                  int64_t sz, int bx, int by) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(nx), static_cast<cuuint64_t>(ny), static_cast<cuuint64_t>(nz)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(sy), static_cast<cuuint64_t>(sz)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(bx), static_cast<cuuint32_t>(by), 1};
  return encode_map(map, type, data, 3, dims, strides, box);
}

// SMs of the current device.
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && known[dev].load(std::memory_order_relaxed) > 0) return known[dev].load(std::memory_order_relaxed);
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace mfr
