// The experts' 16-bit products: rows in expert order times their experts' weights, and the gradients to the rows and to
// the weights, on the fifth-generation tensor cores.
//
// The three directions are one kernel over tiles of the output, D = A * B summed over the reduction:
//   forward          A = rows [r, i]         B = weight [n, i]       over i: both operands' lines run along the reduction
//   gradient to rows A = d_out [r, n]        B = weight [n, i]       over n: B's lines run along its columns i
//   to weights       A = d_out [r, n]        B = rows [r, i]         over the expert's rows r: both along the columns
// The instruction takes either kind of lines, so nothing is transposed in memory.
//
// A persistent CTA (or a pair of CTAs) takes tiles of 128 rows (256) x BN columns.  One warp copies the operands in by
// tensor copies, 64 values of the reduction a stage; one thread issues the matrix instructions into one of two
// accumulators in tensor memory; four warps take finished accumulators out, round and store them meanwhile.
#include "experts_device.cuh"

namespace mfr {

__device__ unsigned int g_expert_wait_timeouts = 0;

namespace {

enum Dir { kForward = 0, kGated = 1, kRowsGrad = 2, kWeightGrad = 3 };

constexpr int kThreads = 256;
constexpr int kEpilogueWarp = 4;                 // first of four
constexpr int kDepth = 64;                       // reduction values of a stage: lines of 128 bytes
constexpr int kTileM = kExpertTileRows;          // rows of A of one CTA
constexpr int kABytes = kTileM * kDepth * 2;
constexpr int kSmallRows = 16;                   // rows of the small box of A
constexpr int kBarBytes = 256;

template <typename T> constexpr bool kIsBf16 = false;
template <> constexpr bool kIsBf16<__nv_bfloat16> = true;

struct Params {
  CUtensorMap a, a_small, b;
  const int32_t* offsets;
  const int32_t* counts;
  int32_t E, R;
  int32_t n_red;       // reduction length (the weights' gradient: the expert's rows)
  int32_t n_m, n_out;  // the weights' gradient: rows of D; columns of D (gated: of the output)
  int32_t tiles_n;     // column tiles
  int32_t tiles_m;     // the weights' gradient: row tiles
  int32_t zero_free, accumulate;
  uint8_t* out;
  int64_t out_stride;  // bytes
  uint8_t* gate_up;
  int64_t gate_up_stride;
};

template <int D, int Ctas, int BN>
struct Shape {
  static constexpr int kBRows = BN / Ctas;  // columns of D whose operand this CTA copies
  static constexpr int kBBytes = kBRows * kDepth * 2;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStage;
  static constexpr bool kALines = D == kWeightGrad;
  static constexpr bool kBLines = D == kRowsGrad || D == kWeightGrad;
  // what one CTA holds besides the stages: the barriers and, but for the weights' gradient, the experts' first tiles
  static constexpr int kFixed = kBarBytes + (D == kWeightGrad ? 0 : (MFR_MAX_EXPERTS + 1 + 33) * 4);
  static constexpr int kSmem = 1024 + kStages * kStage + kFixed;
};

struct Tile {
  int e;      // expert
  int row0;   // first row of D that is a row in expert order (weights' gradient: the expert's first row)
  int left;   // rows of the expert from row0 on
  int m0;     // weights' gradient: first row of D
  int n0;     // first column of D
  int steps;  // stages of the reduction
};

template <int D, int Ctas, int BN>
__device__ __forceinline__ Tile tile_at(const Params& p, const int* first, uint32_t t) {
  Tile x;
  constexpr int kCols = D == kGated ? BN / 2 : BN;
  if constexpr (D == kWeightGrad) {
    const uint32_t per = static_cast<uint32_t>(p.tiles_m) * p.tiles_n;
    x.e = t / per;
    const uint32_t in = t % per;
    x.m0 = in / p.tiles_n * (kTileM * Ctas);
    x.n0 = in % p.tiles_n * kCols;
    const RowSpan s = expert_rows(p.offsets, p.counts, x.e, p.R);
    x.row0 = s.begin;
    x.left = s.end - s.begin;
    x.steps = (x.left + kDepth - 1) / kDepth;
  } else {
    const int m = t / p.tiles_n;
    x.n0 = t % p.tiles_n * kCols;
    x.e = tile_expert(first, p.E, m);
    const RowSpan s = expert_rows(p.offsets, p.counts, x.e, p.R);
    x.row0 = s.begin + (m - first[x.e]) * (kTileM * Ctas);
    x.left = s.end - x.row0;
    x.m0 = 0;
    x.steps = (p.n_red + kDepth - 1) / kDepth;
  }
  return x;
}

template <typename T>
__device__ __forceinline__ void store8(uint8_t* dst, const float v[8]) {
  *reinterpret_cast<uint4*>(dst) = make_uint4(Act<T>::pack(v[0], v[1]), Act<T>::pack(v[2], v[3]), Act<T>::pack(v[4], v[5]), Act<T>::pack(v[6], v[7]));
}

// T: the operands' type; O: that of D (FP32 for the weights' gradient alone).
template <int D, int Ctas, int BN, typename T, typename O>
__global__ void __launch_bounds__(kThreads, 1) expert_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, Ctas, BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  const uint32_t stage0 = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kStages * S::kStage);
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * S::kStages;
  const uint32_t dfull0 = empty0 + 8 * S::kStages, dempty0 = dfull0 + 16, ready = dempty0 + 16;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bars + 2 * S::kStages + 5);
  volatile int* give_up = reinterpret_cast<volatile int*>(tmem_at + 1);
  int* first = reinterpret_cast<int*>(smem + S::kStages * S::kStage + kBarBytes);
  static_assert((2 * S::kStages + 6) * 8 <= kBarBytes, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = Ctas == 2 ? cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(dfull0 + 8 * i, 1);
      mbar_init(dempty0 + 8 * i, 4 * Ctas);
    }
    mbar_init(ready, 1);
    *give_up = 0;
    fence_mbar_init();
    tma_prefetch_map(&p.a);
    tma_prefetch_map(&p.b);
  }
  if (warp == 2) tmem_alloc<Ctas>(smem_addr(tmem_at), 2 * BN);
  pdl_launch_dependents();
  pdl_wait();
  if constexpr (D != kWeightGrad)
    count_tiles(first, first + MFR_MAX_EXPERTS + 1, p.offsets, p.counts, p.E, p.R, kTileM * Ctas);
  tmem_fence_before();
  if constexpr (Ctas == 2) cluster_sync(); else __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t tiles = D == kWeightGrad ? static_cast<uint32_t>(p.E) * p.tiles_m * p.tiles_n : static_cast<uint32_t>(first[p.E]) * p.tiles_n;
  const uint32_t t0 = blockIdx.x / Ctas, dt = gridDim.x / Ctas;

  if (warp == 0) {
    // ---- copies
    if (lane == 0) {
      uint32_t s = 0, phase = 0;
      bool ok = true;
      for (uint32_t t = t0; t < tiles && ok; t += dt) {
        const Tile x = tile_at<D, Ctas, BN>(p, first, t);
        // rows of A behind the expert's end may hold another's: they only make rows of D that are not stored
        const int need = x.left - static_cast<int>(rank) * kTileM;
        const int small = Ctas == 1 && D != kWeightGrad && need <= 64 ? (need + kSmallRows - 1) / kSmallRows : 0;
        const uint32_t bytes = Ctas * (small > 0 ? small * kSmallRows * kDepth * 2 : kABytes) + Ctas * S::kBBytes;
        for (int k = 0; k < x.steps; ++k) {
          if (!(ok = wait_phase(empty0 + 8 * s, phase ^ 1, give_up, &g_expert_wait_timeouts))) break;
          const uint32_t a = stage0 + s * S::kStage, b = a + kABytes;
          uint32_t bar = full0 + 8 * s;
          if (rank == 0) mbar_arrive_expect_tx(bar, bytes);
          if constexpr (Ctas == 2) bar = cluster_addr(bar, 0);
          const int r0 = k * kDepth;
          if constexpr (D == kWeightGrad) {
            for (int i = 0; i < kTileM / 64; ++i)
              tma_load_2d<Ctas>(a + i * 64 * kDepth * 2, &p.a, x.m0 + rank * kTileM + i * 64, x.row0 + r0, bar);
            for (int i = 0; i < S::kBRows / 64; ++i)
              tma_load_2d<Ctas>(b + i * 64 * kDepth * 2, &p.b, x.n0 + rank * S::kBRows + i * 64, x.row0 + r0, bar);
          } else {
            if (small > 0)
              for (int i = 0; i < small; ++i) tma_load_2d<Ctas>(a + i * kSmallRows * kDepth * 2, &p.a_small, r0, x.row0 + i * kSmallRows, bar);
            else
              tma_load_2d<Ctas>(a, &p.a, r0, x.row0 + rank * kTileM, bar);
            if constexpr (D == kForward)
              tma_load_3d<Ctas>(b, &p.b, r0, x.n0 + rank * S::kBRows, x.e, bar);
            else if constexpr (D == kGated)  // half of the tile's columns are the gate's, half the others'
              for (int i = 0; i < 2 / Ctas; ++i)
                tma_load_3d<Ctas>(b + i * (BN / 2) * kDepth * 2, &p.b, r0, x.n0 + (rank + i) * p.n_out, x.e, bar);
            else
              for (int i = 0; i < S::kBRows / 64; ++i)
                tma_load_3d<Ctas>(b + i * 64 * kDepth * 2, &p.b, x.n0 + rank * S::kBRows + i * 64, r0, x.e, bar);
          }
          if (++s == S::kStages) { s = 0; phase ^= 1; }
        }
      }
      if (!ok) {  // copies in flight write this CTA's memory: they get 20 ms to land
        const uint64_t since = global_timer_ns();
        while (global_timer_ns() - since < 20000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ---- matrix instructions
    if (rank == 0 || D == kWeightGrad) {
      constexpr uint32_t idesc = f16_idesc(kIsBf16<T>, S::kALines, S::kBLines, kTileM * Ctas, BN);
      uint32_t s = 0, phase = 0, buf = 0, dphase = 0;
      bool ok = true;
      for (uint32_t t = t0; t < tiles && ok; t += dt) {
        int steps = (p.n_red + kDepth - 1) / kDepth, last = kDepth;
        if constexpr (D == kWeightGrad) {
          const RowSpan r = expert_rows(p.offsets, p.counts, t / (static_cast<uint32_t>(p.tiles_m) * p.tiles_n), p.R);
          steps = (r.end - r.begin + kDepth - 1) / kDepth;
          last = r.end - r.begin - (steps - 1) * kDepth;
          if (steps == 0) continue;
        }
        if (!(ok = __all_sync(0xffffffffu, wait_phase(dempty0 + 8 * buf, dphase ^ 1, give_up, &g_expert_wait_timeouts)))) break;
        tmem_fence_after();
        for (int k = 0; k < steps; ++k) {
          if (!(ok = __all_sync(0xffffffffu, wait_phase(full0 + 8 * s, phase, give_up, &g_expert_wait_timeouts)))) break;
          const uint32_t a = stage0 + s * S::kStage, b = a + kABytes;
          if constexpr (D == kWeightGrad) {
            // the lines behind the expert's last row hold other rows: zeros in both operands (0 * NaN is NaN)
            if (k == steps - 1 && last < kDepth) {
              const int lines = kDepth - last;
              for (int i = lane; i < (kTileM + S::kBRows) / 64 * lines * 8; i += 32) {
                const int block = i / (lines * 8), in = i % (lines * 8);
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a + block * 64 * kDepth * 2 + last * 128 + in * 16), "r"(0) : "memory");
              }
              fence_async_shared();
              __syncwarp();
            }
          }
          tmem_fence_after();
          if (lane == 0) {
            const uint64_t da = S::kALines ? swizzled_desc(a, 1024, 64 * kDepth * 2) : swizzled_desc(a, 1024, 16);
            const uint64_t db = S::kBLines ? swizzled_desc(b, 1024, 64 * kDepth * 2) : swizzled_desc(b, 1024, 16);
#pragma unroll
            for (int i = 0; i < kDepth / 16; ++i)  // 16 values of the reduction: 32 bytes of a line, or 16 lines
              mma_f16<Ctas>(tmem + buf * BN, da + i * (S::kALines ? 128 : 2), db + i * (S::kBLines ? 128 : 2), idesc, (k | i) != 0);
            mma_commit<Ctas>(empty0 + 8 * s);
            if (k == steps - 1) mma_commit<Ctas>(dfull0 + 8 * buf);
          }
          __syncwarp();
          if (++s == S::kStages) { s = 0; phase ^= 1; }
        }
        if (buf ^= 1; buf == 0) dphase ^= 1;
      }
    }
  } else if (warp < kEpilogueWarp) {
    // ---- rows of no expert
    if (D != kWeightGrad && p.zero_free) {
      const int w = blockIdx.x * 2 + warp - 2, nw = gridDim.x * 2;
      zero_free_rows(p.out, p.out_stride, static_cast<int64_t>(p.n_out) * 2, p.offsets, p.counts, p.E, p.R, w, nw);
      if (D == kGated && p.gate_up != nullptr)
        zero_free_rows(p.gate_up, p.gate_up_stride, static_cast<int64_t>(p.n_out) * 4, p.offsets, p.counts, p.E, p.R, w, nw);
    }
  } else {
    // ---- finished accumulators
    const int quarter = warp - kEpilogueWarp;
    uint32_t buf = 0, dphase = 0;
    for (uint32_t t = t0; t < tiles; t += dt) {
      const Tile x = tile_at<D, Ctas, BN>(p, first, t);
      const int r = rank * kTileM + quarter * 32 + lane;
      const bool live = D == kWeightGrad ? x.m0 + r < p.n_m : r < x.left;
      const int64_t row = D == kWeightGrad ? static_cast<int64_t>(x.e) * p.n_m + x.m0 + r : static_cast<int64_t>(x.row0) + r;
      uint8_t* out = p.out + row * p.out_stride;
      const bool some = D != kWeightGrad || x.steps > 0;
      if (some) {
        if (!__all_sync(0xffffffffu, wait_phase(dfull0 + 8 * buf, dphase, give_up, &g_expert_wait_timeouts))) break;
        tmem_fence_after();
      }
      const uint32_t d = tmem + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16);
      constexpr int kCols = D == kGated ? BN / 2 : BN;
#pragma unroll 1
      for (int c = 0; c < kCols; c += 32) {
        uint32_t v[32], u[32];
        if (some) {
          tmem_load32(d + c, v);
          if constexpr (D == kGated) tmem_load32(d + BN / 2 + c, u);
          tmem_wait_load();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        if (live) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            const int n = x.n0 + c + i;
            if (n < p.n_out) {
              float y[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(v[i + j]);
              if constexpr (D == kGated) {
                float z[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] = __uint_as_float(u[i + j]);
                if (p.gate_up != nullptr) {
                  uint8_t* g = p.gate_up + row * p.gate_up_stride;
                  store8<T>(g + static_cast<int64_t>(n) * 2, y);
                  store8<T>(g + (static_cast<int64_t>(p.n_out) + n) * 2, z);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = swiglu(y[j], z[j]);
              }
              if constexpr (sizeof(O) == 4) {
                float4* o = reinterpret_cast<float4*>(out + static_cast<int64_t>(n) * 4);
                float4 lo = make_float4(y[0], y[1], y[2], y[3]), hi = make_float4(y[4], y[5], y[6], y[7]);
                if (p.accumulate) {
                  const float4 a = o[0], b = o[1];
                  lo = make_float4(lo.x + a.x, lo.y + a.y, lo.z + a.z, lo.w + a.w);
                  hi = make_float4(hi.x + b.x, hi.y + b.y, hi.z + b.z, hi.w + b.w);
                }
                o[0] = lo;
                o[1] = hi;
              } else {
                store8<T>(out + static_cast<int64_t>(n) * 2, y);
              }
            }
          }
        }
      }
      if (some) {
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (Ctas == 2) mbar_arrive_cluster(cluster_addr(dempty0 + 8 * buf, 0)); else mbar_arrive(dempty0 + 8 * buf);
        }
        if (buf ^= 1; buf == 0) dphase ^= 1;
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  if constexpr (Ctas == 2) cluster_sync(); else __syncthreads();
  if (warp == 2) {
    tmem_fence_after();
    tmem_free<Ctas>(tmem, 2 * BN);
  }
}

// ------------------------------------------------------------------------------------------------
// Launches
// ------------------------------------------------------------------------------------------------

template <int D, int Ctas, int BN, typename T, typename O>
cudaError_t launch(Params& p, int64_t most_tiles, bool pdl, cudaStream_t stream) {
  using S = Shape<D, Ctas, BN>;
  constexpr auto kern = expert_kernel<D, Ctas, BN, T, O>;
  cudaError_t e = allow_smem<kern>(S::kSmem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count() / Ctas * Ctas;
  if (sms == 0) return cudaErrorInvalidDevice;
  const int64_t want = most_tiles * Ctas;
  return launch_pdl(kern, dim3(static_cast<unsigned>(want < sms ? want : sms)), kThreads, S::kSmem, pdl, stream, p, Ctas);
}

CUtensorMapDataType map_type(int act) { return act == MFR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16; }

template <int D, int Ctas, int BN>
cudaError_t launch_rows(int act, int64_t R, int E, Params& p, bool pdl, cudaStream_t stream) {
  p.tiles_n = (p.n_out + (D == kGated ? BN / 2 : BN) - 1) / (D == kGated ? BN / 2 : BN);
  const int64_t tiles = expert_row_tiles(R, E, kTileM * Ctas) * p.tiles_n;
  return act == MFR_BF16 ? launch<D, Ctas, BN, __nv_bfloat16, __nv_bfloat16>(p, tiles, pdl, stream)
                         : launch<D, Ctas, BN, __half, __half>(p, tiles, pdl, stream);
}

}  // namespace

cudaError_t launch_expert_matmul(const mfr_expert_matmul_args& a, cudaStream_t stream) {
  Params p = {};
  const CUtensorMapDataType type = map_type(a.act_dtype);
  const int wide = a.gated ? 2 * a.n_out : a.n_out;
  constexpr int BN = 256;
  const int b_rows = a.gated ? BN / 2 : BN;
  cudaError_t e = encode_map(&p.a, type, a.rows, a.n_in, a.num_rows, 1, a.rows_stride * 2, 0, kDepth, kTileM, 2);
  if (e == cudaSuccess) e = encode_map(&p.a_small, type, a.rows, a.n_in, a.num_rows, 1, a.rows_stride * 2, 0, kDepth, kSmallRows, 2);
  if (e == cudaSuccess)
    e = encode_map(&p.b, type, a.weight, a.n_in, wide, a.E, a.weight_stride * 2, (a.E > 1 ? a.weight_expert_stride : wide * a.weight_stride) * 2,
                   kDepth, b_rows, 3);
  if (e != cudaSuccess) return e;
  p.offsets = a.expert_offsets;
  p.counts = a.expert_counts;
  p.E = a.E;
  p.R = static_cast<int32_t>(a.num_rows);
  p.n_red = a.n_in;
  p.n_out = a.n_out;
  p.zero_free = (a.flags & MFR_FLAG_ZERO_PADDING) != 0;
  p.out = static_cast<uint8_t*>(a.out);
  p.out_stride = a.out_stride * 2;
  p.gate_up = static_cast<uint8_t*>(a.gate_up);
  p.gate_up_stride = a.gate_up_stride * 2;
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  return a.gated ? launch_rows<kGated, 1, BN>(a.act_dtype, a.num_rows, a.E, p, pdl, stream)
                 : launch_rows<kForward, 1, BN>(a.act_dtype, a.num_rows, a.E, p, pdl, stream);
}

cudaError_t launch_expert_rows_grad(const mfr_expert_matmul_backward_args& a, cudaStream_t stream) {
  Params p = {};
  const CUtensorMapDataType type = map_type(a.act_dtype);
  constexpr int BN = 256;
  cudaError_t e = encode_map(&p.a, type, a.d_out, a.n_out, a.num_rows, 1, a.d_out_stride * 2, 0, kDepth, kTileM, 2);
  if (e == cudaSuccess) e = encode_map(&p.a_small, type, a.d_out, a.n_out, a.num_rows, 1, a.d_out_stride * 2, 0, kDepth, kSmallRows, 2);
  if (e == cudaSuccess)
    e = encode_map(&p.b, type, a.weight, a.n_in, a.n_out, a.E, a.weight_stride * 2,
                   (a.E > 1 ? a.weight_expert_stride : a.n_out * a.weight_stride) * 2, 64, kDepth, 3);
  if (e != cudaSuccess) return e;
  p.offsets = a.expert_offsets;
  p.counts = a.expert_counts;
  p.E = a.E;
  p.R = static_cast<int32_t>(a.num_rows);
  p.n_red = a.n_out;
  p.n_out = a.n_in;
  p.zero_free = (a.flags & MFR_FLAG_ZERO_PADDING) != 0;
  p.out = static_cast<uint8_t*>(a.d_rows);
  p.out_stride = a.d_rows_stride * 2;
  return launch_rows<kRowsGrad, 1, BN>(a.act_dtype, a.num_rows, a.E, p, (a.flags & MFR_FLAG_PDL) != 0, stream);
}

cudaError_t launch_expert_weight_grad(const mfr_expert_matmul_backward_args& a, cudaStream_t stream) {
  const int64_t size = a.d_weight_dtype == MFR_FP32 ? 4 : 2;
  if (a.num_rows == 0)
    return a.accumulate ? cudaSuccess : cudaMemsetAsync(a.d_weight, 0, static_cast<size_t>(a.E) * a.n_out * a.n_in * size, stream);
  Params p = {};
  const CUtensorMapDataType type = map_type(a.act_dtype);
  constexpr int BN = 256;
  cudaError_t e = encode_map(&p.a, type, a.d_out, a.n_out, a.num_rows, 1, a.d_out_stride * 2, 0, 64, kDepth, 2);
  if (e == cudaSuccess) e = encode_map(&p.b, type, a.rows, a.n_in, a.num_rows, 1, a.rows_stride * 2, 0, 64, kDepth, 2);
  if (e != cudaSuccess) return e;
  p.offsets = a.expert_offsets;
  p.counts = a.expert_counts;
  p.E = a.E;
  p.R = static_cast<int32_t>(a.num_rows);
  p.n_m = a.n_out;
  p.n_out = a.n_in;
  p.tiles_m = (a.n_out + kTileM - 1) / kTileM;
  p.tiles_n = (a.n_in + BN - 1) / BN;
  p.accumulate = a.accumulate;
  p.out = static_cast<uint8_t*>(a.d_weight);
  p.out_stride = a.n_in * size;
  const int64_t tiles = static_cast<int64_t>(a.E) * p.tiles_m * p.tiles_n;
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  if (a.d_weight_dtype == MFR_FP32)
    return a.act_dtype == MFR_BF16 ? launch<kWeightGrad, 1, BN, __nv_bfloat16, float>(p, tiles, pdl, stream)
                                   : launch<kWeightGrad, 1, BN, __half, float>(p, tiles, pdl, stream);
  return a.act_dtype == MFR_BF16 ? launch<kWeightGrad, 1, BN, __nv_bfloat16, __nv_bfloat16>(p, tiles, pdl, stream)
                                 : launch<kWeightGrad, 1, BN, __half, __half>(p, tiles, pdl, stream);
}

cudaError_t read_and_reset_expert_timeouts(unsigned int* count) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_expert_wait_timeouts, sizeof(unsigned int));
  if (e != cudaSuccess || *count == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_expert_wait_timeouts, &zero, sizeof(unsigned int));
}

}  // namespace mfr
