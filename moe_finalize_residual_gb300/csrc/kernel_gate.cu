// The elementwise operators between the experts' products: the gradient of the gate, NVFP4 quantisation and its inverse.
// All are bound by memory: every input is read once and every output written once, 32 to 48 bytes a thread in flight.
// A row is taken by `tpr` threads of a CTA (whole warps), so that no thread divides by a row's length.
#include "experts_launch.h"

namespace mfr {
namespace {

struct RowShape {
  int tpr;   // threads a row, a multiple of 32
  int rows;  // rows a CTA
};

// Threads for rows of n items, one item a thread where a CTA holds so many.
RowShape row_shape(int n) {
  RowShape s;
  s.tpr = n < 512 ? (n + 31) / 32 * 32 : 512;
  s.rows = s.tpr < 256 ? 256 / s.tpr : 1;
  return s;
}

// ------------------------------------------------------------------------------------------------
// Gradient of the gate
// ------------------------------------------------------------------------------------------------

struct GateParams {
  const uint8_t* gate_up;
  const uint8_t* d_out;
  const int32_t* row_route;
  uint8_t* d_gate_up;
  uint8_t* out;
  int64_t gate_up_stride, d_out_stride, d_gate_up_stride, out_stride;  // bytes
  int64_t num_rows;
  int32_t vectors;  // of 8 values in a half
  int32_t tpr;
};

template <typename T>
__global__ void __launch_bounds__(512) swiglu_backward_kernel(const __grid_constant__ GateParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.tpr) + threadIdx.x / p.tpr;
  if (row >= p.num_rows) return;
  const bool live = p.row_route == nullptr || p.row_route[row] >= 0;
  const int64_t half = static_cast<int64_t>(p.vectors) * 16;
  for (int v = threadIdx.x % p.tpr; v < p.vectors; v += p.tpr) {
    const int64_t at = static_cast<int64_t>(v) * 16;
    const uint8_t* x = p.gate_up + row * p.gate_up_stride + at;
    const uint4 raw_g = ldg16_if(x, live), raw_u = ldg16_if(x + half, live);
    const uint4 raw_d = ldg16_if(p.d_out + row * p.d_out_stride + at, live && p.d_gate_up != nullptr);
    float g[8], u[8], d[8];
    unpack8<T>(raw_g, g);
    unpack8<T>(raw_u, u);
    unpack8<T>(raw_d, d);
    uint32_t dg[4], du[4], y[4];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float a[2], b[2], c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // the logistic function of g; where exp(-g) is infinite it is 0
        const float s = __frcp_rn(1.0f + __expf(-g[i + j]));
        const float sg = g[i + j] * s;
        a[j] = d[i + j] * u[i + j] * (s * (1.0f + (g[i + j] - sg)));
        b[j] = d[i + j] * sg;
        c[j] = sg * u[i + j];
      }
      dg[i / 2] = Act<T>::pack(a[0], a[1]);
      du[i / 2] = Act<T>::pack(b[0], b[1]);
      y[i / 2] = Act<T>::pack(c[0], c[1]);
    }
    if (p.d_gate_up != nullptr) {
      uint8_t* o = p.d_gate_up + row * p.d_gate_up_stride + at;
      *reinterpret_cast<uint4*>(o) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
      *reinterpret_cast<uint4*>(o + half) = make_uint4(du[0], du[1], du[2], du[3]);
    }
    if (p.out != nullptr) *reinterpret_cast<uint4*>(p.out + row * p.out_stride + at) = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

// ------------------------------------------------------------------------------------------------
// NVFP4
// ------------------------------------------------------------------------------------------------

struct Fp4Params {
  const uint8_t* x;   // quantize: read; dequantize: written
  uint8_t* codes;
  uint8_t* sf;
  const float* scale;
  const int32_t* row_route;
  int64_t x_stride;   // bytes
  int64_t rows;       // of a matrix
  int64_t rows_up;    // with the tiles' last rows
  int64_t total;      // rows_up of all matrices
  int64_t sf_bytes;   // of a matrix
  int32_t H, blocks, blocks_up, layout, tpr, act;
};

// Where this thread's row is: false if it has none.
struct Fp4Row {
  int64_t matrix, m, row;
};
__device__ __forceinline__ bool fp4_row(const Fp4Params& p, Fp4Row& r) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.tpr) + threadIdx.x / p.tpr;
  if (i >= p.total) return false;
  r.matrix = i < p.rows_up ? 0 : i / p.rows_up;
  r.m = i - r.matrix * p.rows_up;
  r.row = r.matrix * p.rows + r.m;
  return true;
}

// A thread takes blocks of 16 values.  The scale's bytes of four neighbouring blocks, one word of a tile, are written by
// one thread.
template <typename T>
__global__ void __launch_bounds__(512) nvfp4_quantize_kernel(const __grid_constant__ Fp4Params p) {
  pdl_launch_dependents();
  pdl_wait();
  Fp4Row r;
  if (!fp4_row(p, r)) return;  // (rows are whole warps')
  const float g = *p.scale;
  const bool real = r.m < p.rows;
  const bool live = real && (p.row_route == nullptr || p.row_route[r.row] >= 0);
  for (int k0 = 0; k0 < p.blocks_up; k0 += p.tpr) {
    const int k = k0 + threadIdx.x % p.tpr;
    const bool here = real && k < p.blocks;
    uint32_t sf = 0;
    if (here) {
      const uint8_t* x = p.x + r.row * p.x_stride + static_cast<int64_t>(k) * 32;
      float v[16];
      unpack8<T>(ldg16_if(x, live), v);
      unpack8<T>(ldg16_if(x + 16, live), v + 8);
      float amax = 0.0f;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        amax = fmaxf(amax, fabsf(v[i]));
        nan |= v[i] != v[i];
      }
      // a block that holds a NaN gets the scale NaN: its codes cannot say so
      sf = nan ? 0x7fu : __nv_cvt_float_to_fp8(__fmul_rn(__fdiv_rn(amax, 6.0f), g), __NV_SATFINITE, __NV_E4M3);
      const float wide = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(sf), __NV_E4M3)));
      const float es = wide == 0.0f ? 0.0f : __fdiv_rn(g, wide);
      uint32_t c[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        c[i / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(__fmul_rn(v[2 * i], es), __fmul_rn(v[2 * i + 1], es)),
                                                                   __NV_E2M1, cudaRoundNearest))
                    << (8 * (i % 4));
      *reinterpret_cast<uint2*>(p.codes + r.row * (p.H / 2) + static_cast<int64_t>(k) * 8) = make_uint2(c[0], c[1]);
    }
    uint8_t* to = p.sf + r.matrix * p.sf_bytes;
    if (p.layout == MFR_SF_ROW_MAJOR) {
      if (here) to[r.m * p.blocks + k] = static_cast<uint8_t>(sf);
    } else {
      sf |= __shfl_down_sync(0xffffffffu, sf, 1) << 8;
      sf |= __shfl_down_sync(0xffffffffu, sf, 2) << 16;
      if ((k & 3) == 0 && k < p.blocks_up) *reinterpret_cast<uint32_t*>(to + sf_offset(r.m, k, p.H, p.layout)) = sf;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(512) nvfp4_dequantize_kernel(const __grid_constant__ Fp4Params p) {
  pdl_launch_dependents();
  pdl_wait();
  Fp4Row r;
  if (!fp4_row(p, r) || r.m >= p.rows) return;
  const float g = *p.scale;
  const bool live = p.row_route == nullptr || p.row_route[r.row] >= 0;
  const uint8_t* from = p.sf + r.matrix * p.sf_bytes;
  for (int k = threadIdx.x % p.tpr; k < p.blocks; k += p.tpr) {
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live) {
      const uint2 c = *reinterpret_cast<const uint2*>(p.codes + r.row * (p.H / 2) + static_cast<int64_t>(k) * 8);
      const uint8_t sf = from[sf_offset(r.m, k, p.H, p.layout)];
      const float es = __fdiv_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(sf, __NV_E4M3))), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t pair = ((i < 4 ? c.x : c.y) >> (8 * (i % 4))) & 0xff;
        const float2 v = __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(pair), __NV_E2M1)));
        w[i] = Act<T>::pack(__fmul_rn(v.x, es), __fmul_rn(v.y, es));
      }
    }
    uint4* o = reinterpret_cast<uint4*>(const_cast<uint8_t*>(p.x) + r.row * p.x_stride + static_cast<int64_t>(k) * 32);
    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

Fp4Params fp4_params(const mfr_nvfp4_args& a, bool padding) {
  Fp4Params p = {};
  const bool tiles = a.sf_layout != MFR_SF_ROW_MAJOR;
  p.x = static_cast<const uint8_t*>(a.x);
  p.codes = static_cast<uint8_t*>(a.codes);
  p.sf = static_cast<uint8_t*>(a.sf);
  p.scale = a.scale;
  p.row_route = a.row_route;
  p.x_stride = a.x_stride * 2;
  p.rows = a.rows;
  p.rows_up = tiles && padding ? (a.rows + 127) / 128 * 128 : a.rows;
  p.total = p.rows_up * a.matrices;
  p.sf_bytes = moe_nvfp4_sf_bytes(1, a.rows, a.H, a.sf_layout);
  p.H = a.H;
  p.blocks = a.H / 16;
  p.blocks_up = tiles && padding ? (p.blocks + 3) / 4 * 4 : p.blocks;
  p.layout = a.sf_layout;
  return p;
}

}  // namespace

cudaError_t launch_swiglu_backward(const mfr_swiglu_backward_args& a, cudaStream_t stream) {
  GateParams p = {};
  p.gate_up = static_cast<const uint8_t*>(a.gate_up);
  p.d_out = static_cast<const uint8_t*>(a.d_out);
  p.row_route = a.row_route;
  p.d_gate_up = static_cast<uint8_t*>(a.d_gate_up);
  p.out = static_cast<uint8_t*>(a.out);
  p.gate_up_stride = a.gate_up_stride * 2;
  p.d_out_stride = a.d_out_stride * 2;
  p.d_gate_up_stride = a.d_gate_up_stride * 2;
  p.out_stride = a.out_stride * 2;
  p.num_rows = a.num_rows;
  p.vectors = a.F / 8;
  const RowShape s = row_shape(p.vectors);
  p.tpr = s.tpr;
  const dim3 grid(static_cast<unsigned>((a.num_rows + s.rows - 1) / s.rows));
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  return a.act_dtype == MFR_BF16 ? launch_pdl(swiglu_backward_kernel<__nv_bfloat16>, grid, s.tpr * s.rows, 0, pdl, stream, p)
                                 : launch_pdl(swiglu_backward_kernel<__half>, grid, s.tpr * s.rows, 0, pdl, stream, p);
}

cudaError_t launch_nvfp4_quantize(const mfr_nvfp4_args& a, cudaStream_t stream) {
  Fp4Params p = fp4_params(a, true);
  const RowShape s = row_shape(p.blocks_up);
  p.tpr = s.tpr;
  const dim3 grid(static_cast<unsigned>((p.total + s.rows - 1) / s.rows));
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  return a.act_dtype == MFR_BF16 ? launch_pdl(nvfp4_quantize_kernel<__nv_bfloat16>, grid, s.tpr * s.rows, 0, pdl, stream, p)
                                 : launch_pdl(nvfp4_quantize_kernel<__half>, grid, s.tpr * s.rows, 0, pdl, stream, p);
}

cudaError_t launch_nvfp4_dequantize(const mfr_nvfp4_args& a, cudaStream_t stream) {
  Fp4Params p = fp4_params(a, false);
  const RowShape s = row_shape(p.blocks);
  p.tpr = s.tpr;
  const dim3 grid(static_cast<unsigned>((p.total + s.rows - 1) / s.rows));
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  return a.act_dtype == MFR_BF16 ? launch_pdl(nvfp4_dequantize_kernel<__nv_bfloat16>, grid, s.tpr * s.rows, 0, pdl, stream, p)
                                 : launch_pdl(nvfp4_dequantize_kernel<__half>, grid, s.tpr * s.rows, 0, pdl, stream, p);
}

}  // namespace mfr
