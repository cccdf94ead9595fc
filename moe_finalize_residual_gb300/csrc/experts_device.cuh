// What the experts' products share: bounded waits, the expert's rows on the device, tensor maps, zeroing of the rows of
// no expert.
#pragma once

#include <cudaTypedefs.h>

#include "experts_launch.h"
#include "gate_device.cuh"
#include "mma_device.cuh"

namespace mfr {

constexpr uint64_t kExpertWaitNs = 2000000000ull;

// Bounded wait on an mbarrier phase: false if the CTA is giving up or the limit (about 2 s) ran out; that is counted, and
// starts the giving up.  Where the wait is for a whole reduction, which may well take longer, `progress` counts its stages, and the
// limit starts again when it changes.
// Ctas 2: of arrivals from both CTAs of a pair.
template <int Ctas>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* give_up, unsigned int* timeouts,
                                           const volatile uint32_t* progress = nullptr) {
  const auto arrived = [&] { return Ctas == 1 ? mbar_try_wait(bar, parity) : mbar_try_wait_cluster(bar, parity); };
  if (arrived()) return true;
  uint64_t t0 = global_timer_ns();
  uint32_t seen = progress != nullptr ? *progress : 0;
  for (uint32_t it = 1;; ++it) {
    if (arrived()) return true;
    if ((it & 15u) == 0) {
      if (*give_up) return false;
      const uint64_t now = global_timer_ns();
      if (progress != nullptr && *progress != seen) {
        seen = *progress;
        t0 = now;
      }
      if (now - t0 > kExpertWaitNs) {
        atomicAdd(timeouts, 1u);
        *give_up = 1;
        return false;
      }
    }
  }
}

// Once a wait has run out: what this CTA's copies and matrix instructions in flight read and write stays theirs for 20 ms, in which
// they end.  By the warps that issued them, before the CTA (of a pair: before both) gives up its memory.
__device__ __forceinline__ void drain(volatile int* give_up) {
  if (!*give_up) return;
  const uint64_t since = global_timer_ns();
  while (global_timer_ns() - since < 20000000ull) __nanosleep(1000);
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

// first[e] = the tiles of `tile` rows of the experts before e, e = 0..E, by all threads of the CTA; `scratch` holds 32 ints.  At most
// `most` of them, what R rows fill (below 2^31): where experts share rows the sums could be E times that.
__device__ __forceinline__ void count_tiles(int* first, int* scratch, const int32_t* offsets, const int32_t* counts, int E, int R, int tile, int most) {
  const int n = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int per = (E + n - 1) / n;
  const auto add = [most](int a, int b) { return static_cast<int>(min(static_cast<uint32_t>(a) + b, static_cast<uint32_t>(most))); };
  const auto tiles = [&](int e) {
    const RowSpan s = expert_rows(offsets, counts, e, R);
    return (s.end - s.begin + tile - 1) / tile;
  };
  int upto = 0;  // the sum up to this thread's experts
  for (int i = 0; i < per; ++i) {
    const int e = t * per + i;
    if (e < E) upto = add(upto, tiles(e));
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto = add(upto, v);
  }
  if (lane == 31) scratch[warp] = upto;
  int at = __shfl_up_sync(0xffffffffu, upto, 1);
  if (lane == 0) at = 0;
  __syncthreads();
  for (int w = 0; w < warp; ++w) at = add(at, scratch[w]);
  for (int i = 0; i < per; ++i) {
    const int e = t * per + i;
    if (e < E) {
      first[e] = at;
      at = add(at, tiles(e));
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

// The rows of tile number m, at most `tile`: an expert's rows in equal parts, a multiple of `unit` but for the last, since a short last
// one would use the weights' copies badly.
struct RowPart {
  int e, row0, rows;  // (rows not positive: the parts before it took all)
};
__device__ __forceinline__ RowPart row_part(const int* first, const int32_t* offsets, const int32_t* counts, int E, int R, int m, int tile, int unit) {
  RowPart x;
  x.e = tile_expert(first, E, m);
  const RowSpan s = expert_rows(offsets, counts, x.e, R);
  const int parts = first[x.e + 1] - first[x.e], n = s.end - s.begin;
  const int equal = static_cast<int>((static_cast<uint32_t>(n) + parts - 1) / parts + unit - 1) / unit * unit;  // (n + parts may pass 2^31)
  const int part = equal < tile ? equal : tile;  // (fewer parts than it takes: experts share rows)
  const int at = (m - first[x.e]) * part;
  x.row0 = s.begin + at;
  x.rows = at < 0 ? 0 : n - at < part ? n - at : part;
  return x;
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

// ------------------------------------------------------------------------------------------------
// Results
// ------------------------------------------------------------------------------------------------

template <typename T> constexpr bool kIsBf16 = false;
template <> constexpr bool kIsBf16<__nv_bfloat16> = true;

template <typename T>
__device__ __forceinline__ T to_act(float v) {
  if constexpr (kIsBf16<T>) return __float2bfloat16_rn(v); else return __float2half_rn(v);
}

// `rows` rows of `Line` bytes, `pitch` bytes apart in shared memory, to rows of an output, by the 128 threads of the epilogue;
// of each row the first `values` values that are there.
template <int Line>
__device__ __forceinline__ void store_rows(uint8_t* out, int64_t stride, const uint8_t* box, int pitch, int rows, int values) {
  constexpr int kPieces = Line / 16;  // threads a row
  const int piece = threadIdx.x % kPieces;
  if (piece * 8 >= values) return;
#pragma unroll
  for (int j = threadIdx.x % 128 / kPieces; j < 32; j += 128 / kPieces)
    if (j < rows) *reinterpret_cast<uint4*>(out + j * stride + piece * 16) = *reinterpret_cast<const uint4*>(box + j * pitch + piece * 16);
}

// Where the products' rows go: strides in bytes, `n` values a row; gate_up may be NULL.
struct RowsOut {
  uint8_t* out;
  int64_t out_stride;
  uint8_t* gate_up;
  int64_t gate_up_stride;
  int32_t n;
};

// Four warps that take finished accumulators out together: kOutGroups of them share a tile, each with a buffer of its own.
constexpr int kOutGroups = 2;
constexpr int kOutBytes = 32 * 128 * 2;  // a buffer: 32 rows of 128 values

// One CTA's part of a finished tile, by the 128 threads of group `group`: 128 lanes of tensor memory at `d` (this warp's
// quarter), the values f0.. of the rows row0 .. row0 + rows_all - 1, a column each, times `alpha`.  Gated, the lanes hold 8 gates,
// their 8 others, and so on.  A thread has one value of 32 rows; through shared memory, where 16 (gated: 8) threads find 16
// bytes each of a row: storing from the registers, 2 bytes a thread, took 10 us a tile of 256 rows, more than most reductions,
// and this 3.4 by one group.  The groups take 32 rows in turn, which gains a tenth where the reduction is short.
template <typename T, bool Gated>
__device__ __forceinline__ void store_tile(uint32_t d, int rows_all, int row0, int f0, float alpha, const RowsOut& to, uint8_t* box, int group) {
  constexpr int kLanes = 128, kLine = (Gated ? kLanes / 2 : kLanes) * 2;  // bytes of a row in this CTA's tile
  const int r = threadIdx.x % kLanes, sync = 1 + group;
  const int64_t at = static_cast<int64_t>(f0) * 2;
#pragma unroll 1
  for (int c = group * 32; c < rows_all; c += kOutGroups * 32) {
    uint32_t w[32];
    tmem_load32(d + c, w);
    tmem_wait_load(w);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]) * alpha;
    const int rows = rows_all - c < 32 ? rows_all - c : 32;
    const int64_t row = static_cast<int64_t>(row0) + c;
    named_sync(sync, 128);  // the buffer's last rows are read
    if constexpr (Gated) {
      // lanes 0..7 of each 16 and 8..15 exchange, and each of the two computes every second row
      const int f = r / 16 * 8 + r % 8;
      const bool upper = (r & 8) != 0;
      if (to.gate_up != nullptr) {
#pragma unroll
        for (int j = 0; j < 32; ++j) reinterpret_cast<T*>(box)[j * kLanes + (upper ? kLanes / 2 : 0) + f] = to_act<T>(v[j]);
        named_sync(sync, 128);
        store_rows<kLine>(to.gate_up + row * to.gate_up_stride + at, to.gate_up_stride, box, 2 * kLine, rows, to.n - f0);
        store_rows<kLine>(to.gate_up + row * to.gate_up_stride + at + static_cast<int64_t>(to.n) * 2, to.gate_up_stride, box + kLine, 2 * kLine, rows,
                          to.n - f0);
        named_sync(sync, 128);
      }
      // (the general form for all of them takes the NVFP4 prompt 776 us for 756; a branch a value the one token's product 35.9 for 35.3)
      bool far = false;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float other = __shfl_xor_sync(0xffffffffu, upper ? v[j] : v[j + 1], 8);
        const float gate = upper ? other : v[j];
        far |= j < rows && gate < kNearGate;
        reinterpret_cast<T*>(box)[(j + (upper ? 1 : 0)) * (kLanes / 2) + f] = to_act<T>(swiglu_near(gate, upper ? v[j + 1] : other));
      }
      if (__any_sync(0xffffffffu, far)) {
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float other = __shfl_xor_sync(0xffffffffu, upper ? v[j] : v[j + 1], 8);
          const float gate = upper ? other : v[j];
          // (only they: a row's results do not depend on its neighbours')
          if (gate < kNearGate) reinterpret_cast<T*>(box)[(j + (upper ? 1 : 0)) * (kLanes / 2) + f] = to_act<T>(swiglu(gate, upper ? v[j + 1] : other));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) reinterpret_cast<T*>(box)[j * kLanes + r] = to_act<T>(v[j]);
    }
    named_sync(sync, 128);
    store_rows<kLine>(to.out + row * to.out_stride + at, to.out_stride, box, kLine, rows, to.n - f0);
  }
}

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
// of `box` values, by default the first 128 bytes, in the 128-byte swizzle; what lies outside reads as zeros.
inline cudaError_t encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* data, int rank, const cuuint64_t* dims,
                              const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const auto f = tensor_map_encoder();
  if (f == nullptr) return cudaErrorNotSupported;
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  const CUresult r = f(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(data), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

// The same, gated: `n` gates' rows and `n` others an expert, n a multiple of 8, in boxes of 8 and 8 rows alternately, 128 in all.
inline cudaError_t encode_gated_weights(CUtensorMap* map, CUtensorMapDataType type, const void* data, int64_t nx, int64_t n, int64_t nz, int64_t sy,
                                        int64_t sz, int bx) {
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(nx), 8, 2, static_cast<cuuint64_t>(n / 8), static_cast<cuuint64_t>(nz)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(sy), static_cast<cuuint64_t>(n * sy), static_cast<cuuint64_t>(8 * sy),
                                 static_cast<cuuint64_t>(sz)};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(bx), 8, 2, 8, 1};
  return encode_map(map, type, data, 5, dims, strides, box);
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
