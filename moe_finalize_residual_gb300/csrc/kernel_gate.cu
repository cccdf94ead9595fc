// The elementwise operators between the experts' products: the gradient of the gate, NVFP4 quantisation and its inverse.
// All are bound by memory: every input is read once and every output written once, 32 to 48 bytes a thread in flight.
// A row is taken by `tpr` threads of a CTA (whole warps), so that no thread divides by a row's length.
// Measured on GB300, 32768 rows: the gate's gradient of 2048 values 123 us (0.96 of the copy bandwidth); 7168 values to NVFP4 112 us
// and back 110 (floor 89 each), both held up by their instructions.
#include "experts_device.cuh"

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

// ldg16_if for memory that this kernel may write: an output may be its input.  (As plain loads in a branch: 134 us for 123.)
__device__ __forceinline__ uint4 load16_if(const uint8_t* p, bool on) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
      " @q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p), "r"(static_cast<int>(on)));
  return v;
}

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
    const uint4 raw_g = load16_if(x, live), raw_u = load16_if(x + half, live);
    const uint4 raw_d = load16_if(p.d_out + row * p.d_out_stride + at, live && p.d_gate_up != nullptr);
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
        const float G = g[i + j], U = u[i + j], D = d[i + j];
        const Logistic p = logistic(G);
        const float sg = G * p.m * p.r;  // (times m: g / (1 + exp(-g)))
        a[j] = scaled_product(D, U, p.m, p.m * (p.r * (1.0f + (G - sg * p.m))));
        b[j] = sg * (D * p.m);
        c[j] = sg * (U * p.m);
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

constexpr int kPieces = 4;           // of 8 values, that a thread has in flight
constexpr int kFp4BlocksPerSm = 8;   // at most: some turns of the CTAs that an SM holds at once

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
  int32_t H, blocks, blocks_up, layout, tpr;
};

// Row i of all matrices'; `real` false behind a matrix's last row, `live` false for a row of no route too.
struct Fp4Row {
  int64_t matrix, m, row;
  bool real, live;
};
__device__ __forceinline__ Fp4Row fp4_row(const Fp4Params& p, int64_t i) {
  Fp4Row r;
  r.matrix = i < p.rows_up ? 0 : i / p.rows_up;
  r.m = i - r.matrix * p.rows_up;
  r.row = r.matrix * p.rows + r.m;
  r.real = r.m < p.rows;
  r.live = r.real && (p.row_route == nullptr || p.row_route[r.row] >= 0);
  return r;
}

// Bytes into a matrix's scales of block k of a row: row_at(m) + block_at(k).
__device__ __forceinline__ int64_t row_at(const Fp4Params& p, int64_t m) {
  return p.layout == MFR_SF_ROW_MAJOR ? m * p.blocks : (m >> 7) * (static_cast<int64_t>((p.blocks + 3) >> 2) * 512) + (m & 31) * 16 + (m >> 5 & 3) * 4;
}
__device__ __forceinline__ int block_at(const Fp4Params& p, int k) { return p.layout == MFR_SF_ROW_MAJOR ? k : (k >> 2) * 512 + (k & 3); }

// Eight E2M1 codes, nearest even, at most 6; the even value of a pair in the low half of its byte.
__device__ __forceinline__ uint32_t to_e2m1x8(const float2 v[4]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}

// The largest magnitude of 8 values as they are stored, a NaN's bits if there is one: magnitudes order as their bits.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t largest(uint4 a) {
  const uint32_t m = max_u16x2(max_u16x2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), max_u16x2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// A thread takes 8 values, two neighbouring ones a block, and four of its row's pieces at once.  Whole sectors go each way:
// a block a thread, 32 bytes apart, was slower (H = 7168, 32768 rows: 210 us; with two rows a thread 134; two pieces a thread 132; 112 so).  The scale's bytes of four neighbouring
// blocks, one word of a tile, are written by one thread.
template <typename T>
__global__ void __launch_bounds__(512) nvfp4_quantize_kernel(const __grid_constant__ Fp4Params p) {
  pdl_launch_dependents();
  pdl_wait();
  const float g = *p.scale;
  const int lane_k = threadIdx.x % p.tpr, per = blockDim.x / p.tpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  int64_t i = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / p.tpr;  // (rows are whole warps')
  int base = 0;
  if (i >= p.total) return;
  Fp4Row r = fp4_row(p, i);
  uint4 a[kPieces];
  const auto load = [&](uint4 v[kPieces], const Fp4Row& row, int k0) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) v[u] = ldg16_if(p.x + row.row * p.x_stride + (k0 + u * p.tpr) * 16, row.live && k0 + u * p.tpr < 2 * p.blocks);
  };
  load(a, r, lane_k);
  while (true) {
    // the next pieces' loads are in flight while these are worked on
    int64_t next = i;
    int next_base = base + kPieces * p.tpr;
    if (next_base >= 2 * p.blocks_up) next_base = 0, next += step;
    const bool more = next < p.total;
    Fp4Row r1 = r;
    uint4 a1[kPieces];
    if (more) {
      if (next != i) r1 = fp4_row(p, next);
      load(a1, r1, next_base + lane_k);
    }
    const int k0 = base + lane_k;
    uint8_t* codes = p.codes + r.row * (p.H / 2);
    uint8_t* to = p.sf + r.matrix * p.sf_bytes + row_at(p, r.m);
    const bool odd = (threadIdx.x & 1) != 0;
#pragma unroll
    for (int v = 0; v < kPieces; v += 2) {
      // of two neighbouring threads one finds the scale of their first block, the other that of their second
      uint32_t top = largest(a[v]), top1 = largest(a[v + 1]);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top1 = max(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
      const float amax = Act<T>::unpack(odd ? top1 : top).x;
      // a block that holds a NaN gets the scale NaN: its codes cannot say so
      uint32_t found = amax != amax ? 0x7fu : __nv_cvt_float_to_fp8(__fmul_rn(__fdiv_rn(amax, 6.0f), g), __NV_SATFINITE, __NV_E4M3);
      if (!r.real || k0 + (odd ? v + 1 : v) * p.tpr >= 2 * p.blocks) found = 0;
      const float wide = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(found), __NV_E4M3)));
      const float inverse = wide == 0.0f ? 0.0f : __fdiv_rn(g, wide);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = k0 + (v + u) * p.tpr;
        const bool here = r.real && k < 2 * p.blocks;
        uint32_t sf = __shfl_sync(0xffffffffu, found, u, 2);
        const float es = __shfl_sync(0xffffffffu, inverse, u, 2);
        const float2 es2 = make_float2(es, es);
        const uint32_t w[4] = {a[v + u].x, a[v + u].y, a[v + u].z, a[v + u].w};
        float2 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = __fmul2_rn(Act<T>::unpack(w[j]), es2);
        if (here) *reinterpret_cast<uint32_t*>(codes + k * 4) = to_e2m1x8(y);
        if (p.layout == MFR_SF_ROW_MAJOR) {
          if (here && (k & 1) == 0) to[k >> 1] = static_cast<uint8_t>(sf);
        } else {
          sf |= __shfl_down_sync(0xffffffffu, sf, 2) << 8;
          sf |= __shfl_down_sync(0xffffffffu, sf, 4) << 16;
          if ((k & 7) == 0 && k < 2 * p.blocks_up) *reinterpret_cast<uint32_t*>(to + block_at(p, k >> 1)) = sf;
        }
      }
    }
    if (!more) break;
    i = next;
    base = next_base;
    r = r1;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) a[u] = a1[u];
  }
}

// The values of four codes, in FP16, which holds them exactly.
__device__ __forceinline__ void from_e2m1x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b8 b0, b1;\n .reg .b16 w;\n cvt.u16.u32 w, %2;\n mov.b16 {b0, b1}, w;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

template <typename T>
__global__ void __launch_bounds__(512) nvfp4_dequantize_kernel(const __grid_constant__ Fp4Params p) {
  pdl_launch_dependents();
  pdl_wait();
  const float g = *p.scale;
  const int lane_k = threadIdx.x % p.tpr, per = blockDim.x / p.tpr;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / p.tpr; i < p.total; i += static_cast<int64_t>(gridDim.x) * per) {
    const Fp4Row r = fp4_row(p, i);
    const uint8_t* codes = p.codes + r.row * (p.H / 2);
    const uint8_t* from = p.sf + r.matrix * p.sf_bytes + row_at(p, r.m);
    uint8_t* x = const_cast<uint8_t*>(p.x) + r.row * p.x_stride;
    for (int base = 0; base < 2 * p.blocks; base += kPieces * p.tpr) {  // (by whole warps, for the shuffles)
      const int k0 = base + lane_k;
      uint32_t c[kPieces], sf[kPieces];
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int k = k0 + u * p.tpr;
        const bool here = r.live && k < 2 * p.blocks;
        c[u] = here ? __ldg(reinterpret_cast<const uint32_t*>(codes + k * 4)) : 0;
        sf[u] = here ? __ldg(from + block_at(p, k >> 1)) : 0;
      }
#pragma unroll
      for (int v = 0; v < kPieces; v += 2) {
        // (one division for the two blocks of two neighbouring threads)
        const uint32_t of = (threadIdx.x & 1) != 0 ? sf[v + 1] : sf[v];
        const float quotient = __fdiv_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(of), __NV_E4M3))), g);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int k = k0 + (v + u) * p.tpr;
          const float es = __shfl_sync(0xffffffffu, quotient, u, 2);
          const float2 es2 = make_float2(es, es);
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t h[2];
            from_e2m1x4(c[v + u] >> (16 * i), h[0], h[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 y = __fmul2_rn(Act<__half>::unpack(h[j]), es2);
              w[2 * i + j] = Act<T>::pack(y.x, y.y);
            }
          }
          if (k < 2 * p.blocks) *reinterpret_cast<uint4*>(x + k * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
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

// CTAs that stay for several rows: what a thread works out once (the divisions above all) is a third of its instructions when
// it has one row.
dim3 fp4_grid(const Fp4Params& p, const RowShape& s) {
  const int64_t all = (p.total + s.rows - 1) / s.rows, most = int64_t{kFp4BlocksPerSm} * sm_count();
  return dim3(static_cast<unsigned>(all < most || most == 0 ? all : most));
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
  const RowShape s = row_shape((2 * p.blocks_up + kPieces - 1) / kPieces);
  p.tpr = s.tpr;
  const dim3 grid = fp4_grid(p, s);
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  return a.act_dtype == MFR_BF16 ? launch_pdl(nvfp4_quantize_kernel<__nv_bfloat16>, grid, s.tpr * s.rows, 0, pdl, stream, p)
                                 : launch_pdl(nvfp4_quantize_kernel<__half>, grid, s.tpr * s.rows, 0, pdl, stream, p);
}

cudaError_t launch_nvfp4_dequantize(const mfr_nvfp4_args& a, cudaStream_t stream) {
  Fp4Params p = fp4_params(a, false);
  const RowShape s = row_shape((2 * p.blocks + kPieces - 1) / kPieces);
  p.tpr = s.tpr;
  const dim3 grid = fp4_grid(p, s);
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  return a.act_dtype == MFR_BF16 ? launch_pdl(nvfp4_dequantize_kernel<__nv_bfloat16>, grid, s.tpr * s.rows, 0, pdl, stream, p)
                                 : launch_pdl(nvfp4_dequantize_kernel<__half>, grid, s.tpr * s.rows, 0, pdl, stream, p);
}

}  // namespace mfr
