// Rows in and out of expert order: the dispatch of token rows to the expert-sorted rows, and the gradient
// of the finalize to those rows and to the expert scales.
//
// Both move whole 16-byte vectors and are bound by HBM: a token's row is read once (K rows are written
// from it), every expert row once.  A CTA takes one token (or a slice of its row) and, in the gradient, up to
// KB of its routes, so that all its row vectors are in flight together; rows that no route names are set to
// zero by the CTAs behind the tokens'.
//
// Measured on GB300 (copy bandwidth 6779 GB/s): dispatch of 4096 tokens of 7168 FP16 elements to 8 experts, a
// quarter of the routes masked, 529 MB in 82 us (0.95 of the copy); the gradient of the same batch in BF16, 881 MB
// in 132 us (0.98).
#include "layer_launch.h"

namespace mfr {
namespace {

constexpr int kZeroRows = 8;  // rows looked at by one CTA of the zeroing part of a grid

__device__ __forceinline__ void stg16(uint8_t* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

// Sets the rows without a route among rows [first, first + kZeroRows) to zero.
__device__ __forceinline__ void zero_rows(const int32_t* row_route, int64_t first, int64_t num_rows, uint8_t* rows, int64_t row_bytes) {
  for (int i = 0; i < kZeroRows; ++i) {
    const int64_t r = first + i;
    if (r >= num_rows) return;
    if (row_route[r] >= 0) continue;
    for (int64_t b = threadIdx.x * 16; b < row_bytes; b += blockDim.x * 16) stg16(rows + r * row_bytes + b, make_uint4(0, 0, 0, 0));
  }
}

struct RowsGrid {
  int slices;        // CTAs a token
  int64_t token_ctas;
  int64_t zero_ctas;
};

// ---------------------------------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------------------------------

struct DispatchParams {
  mfr_dispatch_args a;
  RowsGrid g;
  int slice_vec;  // 16-byte vectors of a slice
};

// CTA (token, slice): reads the slice of x[t] once and writes it to each of the token's rows.
__global__ void __launch_bounds__(512) dispatch_kernel(const __grid_constant__ DispatchParams p) {
  __shared__ int64_t dst[MFR_MAX_TOP_K];
  const mfr_dispatch_args& a = p.a;
  uint8_t* rows = static_cast<uint8_t*>(a.rows);
  pdl_launch_dependents();
  pdl_wait();
  const int64_t cta = blockIdx.x;
  if (cta >= p.g.token_ctas) {
    zero_rows(a.row_route, (cta - p.g.token_ctas) * kZeroRows, a.num_rows, rows, a.row_bytes);
    return;
  }
  const int64_t t = cta / p.g.slices;
  const int slice = static_cast<int>(cta % p.g.slices);
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    const int64_t r = a.perm_idx[t * a.K + k];
    dst[k] = r >= 0 && r < a.num_rows ? r * a.row_bytes : -1;
  }
  const int nvec = static_cast<int>(a.row_bytes / 16);
  const int v0 = slice * p.slice_vec, v1 = min(nvec, v0 + p.slice_vec);
  const uint8_t* src = static_cast<const uint8_t*>(a.x) + t * a.row_bytes;
  int v = v0 + threadIdx.x;
  uint4 val = make_uint4(0, 0, 0, 0);
  if (v < v1) val = ldg16(src + static_cast<int64_t>(v) * 16);
  __syncthreads();
  while (v < v1) {
    for (int k = 0; k < a.K; ++k)
      if (dst[k] >= 0) stg16(rows + dst[k] + static_cast<int64_t>(v) * 16, val);
    v += blockDim.x;
    if (v < v1) val = ldg16(src + static_cast<int64_t>(v) * 16);
  }
}

// ---------------------------------------------------------------------------------------------------
// Gradient of the finalize
// ---------------------------------------------------------------------------------------------------

constexpr int kBackThreads = 256;

struct RoutedBackwardParams {
  mfr_routed_backward_args a;
  RowsGrid g;
};

// CTA (token, KB of its routes): the routes' rows stream past the token's gradient once, giving the dot
// products and the gradient rows.  The dot products meet by a warp butterfly, then over the warps in order.
template <typename A, int KB>
__global__ void __launch_bounds__(kBackThreads) routed_backward_kernel(const __grid_constant__ RoutedBackwardParams p) {
  __shared__ int64_t at[KB];
  __shared__ float weight[KB];
  __shared__ float part[kBackThreads / 32][KB];
  const mfr_routed_backward_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row_bytes = static_cast<int64_t>(a.H) * 2;
  uint8_t* d_rows = static_cast<uint8_t*>(a.d_gemm2);
  const uint8_t* rows = static_cast<const uint8_t*>(a.gemm2_out);
  pdl_launch_dependents();
  pdl_wait();
  const int64_t cta = blockIdx.x;
  if (cta >= p.g.token_ctas) {
    zero_rows(a.row_route, (cta - p.g.token_ctas) * kZeroRows, a.num_rows, d_rows, row_bytes);
    return;
  }
  const int64_t t = cta / p.g.slices;
  const int k0 = static_cast<int>(cta % p.g.slices) * KB;
  if (tid < KB) {
    const int k = k0 + tid;
    int64_t r = k < a.K ? a.perm_idx[t * a.K + k] : -1;
    if (r >= a.num_rows) r = -1;
    at[tid] = r < 0 ? -1 : r * row_bytes;
    weight[tid] = r < 0 ? 0.0f : __fmul_rn(load_scale(a.expert_scale, t * a.K + k, a.scale_dtype), a.routed_scaling_factor);
  }
  __syncthreads();
  float acc[KB];
#pragma unroll
  for (int i = 0; i < KB; ++i) acc[i] = 0.0f;
  const uint8_t* d_out = static_cast<const uint8_t*>(a.d_out) + t * row_bytes;
  const bool dots = a.d_scale != nullptr;
  for (int64_t b = tid * 16; b < row_bytes; b += kBackThreads * 16) {
    float d[8];
    uint4 x[KB];
    const uint4 raw = ldg16(d_out + b);
    if (dots) {
#pragma unroll
      for (int i = 0; i < KB; ++i) x[i] = ldg16_if(rows + at[i] + b, at[i] >= 0);
    }
    unpack8<A>(raw, d);
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      if (at[i] < 0) continue;
      if (dots) {
        float v[8];
        unpack8<A>(x[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i] = __fmaf_rn(v[j], d[j], acc[i]);
      }
      if (d_rows != nullptr) {
        const float w = weight[i];
        stg16(d_rows + at[i] + b, make_uint4(Act<A>::pack(d[0] * w, d[1] * w), Act<A>::pack(d[2] * w, d[3] * w),
                                             Act<A>::pack(d[4] * w, d[5] * w), Act<A>::pack(d[6] * w, d[7] * w)));
      }
    }
  }
  if (!dots) return;
#pragma unroll
  for (int i = 0; i < KB; ++i) {
    const float s = warp_sum(acc[i]);
    if (lane == 0) part[warp][i] = s;
  }
  __syncthreads();
  if (tid < KB && k0 + tid < a.K) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kBackThreads / 32; ++w) s += part[w][tid];
    s = at[tid] < 0 ? 0.0f : s * a.routed_scaling_factor;
    const int64_t i = t * a.K + k0 + tid;
    if (a.scale_dtype == MFR_FP32)
      static_cast<float*>(a.d_scale)[i] = s;
    else if (a.scale_dtype == MFR_BF16)
      static_cast<__nv_bfloat16*>(a.d_scale)[i] = __float2bfloat16_rn(s);
    else
      static_cast<__half*>(a.d_scale)[i] = __float2half_rn(s);
  }
}

template <typename A>
cudaError_t launch_routed_backward_t(const mfr_routed_backward_args& a, cudaStream_t stream) {
  RoutedBackwardParams p{a, {}};
  // Up to 8 routes a CTA, so that a thread has as many rows in flight and reads the token's gradient once, as long as
  // that leaves three CTAs for each SM.  us at KB = 1 / 2 / 4 / 8: 8 tokens of H 7168, top-8, 3.2 / 3.5 / 4.1 / 5.6; 64
  // tokens of H 3584, top-16, 4.6 / 4.3 / 4.7 / 6.6; 152 of them 7.9 / 6.5 / 5.7 / 6.1; 4096 tokens of H 7168, top-8,
  // 191 / 149 / 134 / 133.
  int kb = 1;
  while (kb < 8 && kb < a.K && static_cast<int64_t>(a.T) * ((a.K + 2 * kb - 1) / (2 * kb)) >= 3 * 152) kb *= 2;
  p.g.slices = (a.K + kb - 1) / kb;
  p.g.token_ctas = static_cast<int64_t>(a.T) * p.g.slices;
  p.g.zero_ctas = a.row_route != nullptr && a.d_gemm2 != nullptr ? (a.num_rows + kZeroRows - 1) / kZeroRows : 0;
  const int64_t grid = p.g.token_ctas + p.g.zero_ctas;
  if (grid == 0) return cudaSuccess;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  const bool pdl = a.flags & MFR_FLAG_PDL;
  const dim3 g(static_cast<unsigned>(grid));
  switch (kb) {
    case 1: return launch_pdl<RoutedBackwardParams>(routed_backward_kernel<A, 1>, g, kBackThreads, 0, pdl, stream, p);
    case 2: return launch_pdl<RoutedBackwardParams>(routed_backward_kernel<A, 2>, g, kBackThreads, 0, pdl, stream, p);
    case 4: return launch_pdl<RoutedBackwardParams>(routed_backward_kernel<A, 4>, g, kBackThreads, 0, pdl, stream, p);
    default: return launch_pdl<RoutedBackwardParams>(routed_backward_kernel<A, 8>, g, kBackThreads, 0, pdl, stream, p);
  }
}

}  // namespace

cudaError_t launch_dispatch(const mfr_dispatch_args& a, cudaStream_t stream) {
  DispatchParams p{a, {}, 0};
  const int nvec = static_cast<int>(a.row_bytes / 16);
  // Whole rows a CTA for batches that fill the SMs four times, else slices of at least one warp's vectors.  With one
  // CTA an SM in place of four: 300 tokens of 6144 BF16 elements, top-8, 10.0 us against 6.1; 16 tokens 1.9 either way.
  int64_t slices = a.T > 0 ? (4 * 152 + a.T - 1) / a.T : 1;
  const int most = (nvec + 31) / 32;
  if (slices > most) slices = most;
  const int per = ((nvec + static_cast<int>(slices) - 1) / static_cast<int>(slices) + 31) / 32 * 32;
  p.slice_vec = per;
  p.g.slices = (nvec + per - 1) / per;
  p.g.token_ctas = static_cast<int64_t>(a.T) * p.g.slices;
  p.g.zero_ctas = a.row_route != nullptr ? (a.num_rows + kZeroRows - 1) / kZeroRows : 0;
  const int64_t grid = p.g.token_ctas + p.g.zero_ctas;
  if (grid == 0) return cudaSuccess;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  // threads: the slice in as few rounds as 512 threads need, evenly
  const int rounds = (per + 511) / 512;
  const int block = ((per + rounds - 1) / rounds + 31) / 32 * 32;
  return launch_pdl<DispatchParams>(dispatch_kernel, dim3(static_cast<unsigned>(grid)), block, 0, a.flags & MFR_FLAG_PDL, stream, p);
}

cudaError_t launch_routed_backward(const mfr_routed_backward_args& a, cudaStream_t stream) {
  return a.act_dtype == MFR_BF16 ? launch_routed_backward_t<__nv_bfloat16>(a, stream)
                                 : launch_routed_backward_t<__half>(a, stream);
}

}  // namespace mfr
