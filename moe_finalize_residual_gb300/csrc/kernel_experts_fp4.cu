// The experts' NVFP4 product: rows in expert order times their experts' weights, both as E2M1 codes with an E4M3 scale for
// every 16 values, on the fifth-generation tensor cores, which take codes and scales as they are.
//
// The kernel is that of the 16-bit products (kernel_experts.cu): persistent CTAs, tiles of 128 rows x 256 columns, operands by
// tensor copies, the accumulator in tensor memory.  A stage is 256 values of the reduction.  The weights' scales lie in the
// tiles that tensor memory wants and are copied as they are; the rows' scales are row-major (rows begin anywhere), so four
// warps, a stage each in turn, put them into that order on their way through shared memory.
#include "experts_device.cuh"

namespace mfr {

__device__ unsigned int g_expert_nvfp4_wait_timeouts = 0;

namespace {

constexpr int kThreads = 384;
constexpr int kEpilogueWarp = 4;  // first of four
constexpr int kScaleWarp = 8;     // first of four
constexpr int kDepth = 256;       // reduction values of a stage: lines of 128 bytes
constexpr int kTileM = kExpertTileRows;
constexpr int kTileN = 256;
constexpr int kABytes = kTileM * kDepth / 2;
constexpr int kBBytes = kTileN * kDepth / 2;
constexpr int kSfaBytes = kTileM * kDepth / 16;
constexpr int kSfbBytes = kTileN * kDepth / 16;
constexpr int kStage = kABytes + kBBytes + kSfaBytes + kSfbBytes;
constexpr int kStages = 4;
constexpr int kSmallRows = 16;
constexpr int kBarBytes = 256;
constexpr int kSmem = 1024 + kStages * kStage + kBarBytes + (MFR_MAX_EXPERTS + 1 + 33) * 4;
constexpr uint32_t kSfColumn = 256;                          // tensor-memory columns: D, then the stages' scales
constexpr uint32_t kSfColumns = (kSfaBytes + kSfbBytes) / 128;  // of a stage: 4 bytes a lane and column
static_assert(kSfColumn + kStages * kSfColumns <= 512, "tensor memory");

struct Params {
  CUtensorMap a, a_small, b;
  const int32_t* offsets;
  const int32_t* counts;
  const uint8_t* sf;         // rows' scales, row-major
  const uint8_t* weight_sf;  // weights' scales in tiles
  const float* alpha;
  int32_t E, R;
  int32_t n_in, n_out;
  int32_t tiles_n;
  int32_t sf_tiles;          // tiles of 128 weight rows an expert
  int32_t zero_free;
  uint8_t* out;
  int64_t out_stride;        // bytes
};

struct Tile {
  int e, row0, left, n0;
};

template <bool Gated>
__device__ __forceinline__ Tile tile_at(const Params& p, const int* first, uint32_t t) {
  Tile x;
  const int m = t / p.tiles_n;
  x.n0 = t % p.tiles_n * (Gated ? kTileN / 2 : kTileN);
  x.e = tile_expert(first, p.E, m);
  const RowSpan s = expert_rows(p.offsets, p.counts, x.e, p.R);
  x.row0 = s.begin + (m - first[x.e]) * kTileM;
  x.left = s.end - x.row0;
  return x;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

template <bool Gated, typename T>
__global__ void __launch_bounds__(kThreads, 1) expert_nvfp4_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  const uint32_t stage0 = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStage);
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * kStages, dfull = empty0 + 8 * kStages, dempty = dfull + 8;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 2);
  volatile int* give_up = reinterpret_cast<volatile int*>(tmem_at + 1);
  int* first = reinterpret_cast<int*>(smem + kStages * kStage + kBarBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned int* const timeouts = &g_expert_nvfp4_wait_timeouts;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 2);  // the copies' bytes, and the rows' scales
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(dfull, 1);
    mbar_init(dempty, 4);
    *give_up = 0;
    fence_mbar_init();
    tma_prefetch_map(&p.a);
    tma_prefetch_map(&p.b);
  }
  if (warp == 2) tmem_alloc<1>(smem_addr(tmem_at), 512);
  pdl_launch_dependents();
  pdl_wait();
  count_tiles(first, first + MFR_MAX_EXPERTS + 1, p.offsets, p.counts, p.E, p.R, kTileM);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t tiles = static_cast<uint32_t>(first[p.E]) * p.tiles_n;
  const int steps = (p.n_in + kDepth - 1) / kDepth;
  const int chunks = p.n_in / 64;  // instructions a tile, and columns of 512 bytes of the scales' tiles

  if (warp == 0) {
    // ---- copies
    if (lane == 0) {
      uint32_t s = 0, phase = 0;
      bool ok = true;
      for (uint32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const Tile x = tile_at<Gated>(p, first, t);
        const int small = x.left <= 64 ? (x.left + kSmallRows - 1) / kSmallRows : 0;
        const int sf0 = x.n0 / 128, sf1 = Gated ? (p.n_out + x.n0) / 128 : sf0 + 1;
        const int n_sf = sf1 < p.sf_tiles ? 2 : 1;  // (the last tile of columns may hold 128 of them)
        const uint8_t* wsf = p.weight_sf + static_cast<int64_t>(x.e) * p.sf_tiles * chunks * 512;
        for (int k = 0; k < steps; ++k) {
          if (!(ok = wait_phase(empty0 + 8 * s, phase ^ 1, give_up, timeouts))) break;
          const uint32_t a = stage0 + s * kStage, b = a + kABytes, sfb = b + kBBytes + kSfaBytes, bar = full0 + 8 * s;
          const int n = chunks - 4 * k < 4 ? chunks - 4 * k : 4;
          mbar_arrive_expect_tx(bar, (small > 0 ? small * kSmallRows * 128 : kABytes) + kBBytes + n_sf * n * 512);
          if (small > 0)
            for (int i = 0; i < small; ++i) tma_load_2d<1>(a + i * kSmallRows * 128, &p.a_small, k * 128, x.row0 + i * kSmallRows, bar);
          else
            tma_load_2d<1>(a, &p.a, k * 128, x.row0, bar);
          if constexpr (Gated) {
            tma_load_3d<1>(b, &p.b, k * 128, x.n0, x.e, bar);
            tma_load_3d<1>(b + kBBytes / 2, &p.b, k * 128, p.n_out + x.n0, x.e, bar);
          } else {
            tma_load_3d<1>(b, &p.b, k * 128, x.n0, x.e, bar);
          }
          bulk_load(sfb, wsf + (static_cast<int64_t>(sf0) * chunks + 4 * k) * 512, n * 512, bar);
          if (n_sf == 2) bulk_load(sfb + 2048, wsf + (static_cast<int64_t>(sf1) * chunks + 4 * k) * 512, n * 512, bar);
          if (++s == kStages) { s = 0; phase ^= 1; }
        }
      }
      if (!ok) {  // copies in flight write this CTA's memory: they get 20 ms to land
        const uint64_t since = global_timer_ns();
        while (global_timer_ns() - since < 20000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ---- matrix instructions
    if (lane == 0) {
      constexpr uint32_t idesc = nvfp4_idesc(kTileM, kTileN);
      uint32_t s = 0, phase = 0, dphase = 0;
      bool ok = true;
      for (uint32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        if (!(ok = wait_phase(dempty, dphase ^ 1, give_up, timeouts))) break;
        tmem_fence_after();
        for (int k = 0; k < steps; ++k) {
          if (!(ok = wait_phase(full0 + 8 * s, phase, give_up, timeouts))) break;
          tmem_fence_after();
          const uint32_t a = stage0 + s * kStage, b = a + kABytes, sfa = b + kBBytes, sfb = sfa + kSfaBytes;
          const uint64_t da = swizzled_desc(a, 1024, 16), db = swizzled_desc(b, 1024, 16);
          const uint32_t ta = tmem + kSfColumn + s * kSfColumns, tb = ta + kSfaBytes / 128;
          const int n = chunks - 4 * k < 4 ? chunks - 4 * k : 4;
          for (int i = 0; i < n; ++i) {
            tmem_copy_scales<1>(ta + 4 * i, sfa + 512 * i);
            tmem_copy_scales<1>(tb + 8 * i, sfb + 512 * i);
            tmem_copy_scales<1>(tb + 8 * i + 4, sfb + 2048 + 512 * i);
          }
          for (int i = 0; i < n; ++i) mma_nvfp4<1>(tmem, da + 2 * i, db + 2 * i, idesc, ta + 4 * i, tb + 8 * i, (k | i) != 0);
          mma_commit<1>(empty0 + 8 * s);
          if (k == steps - 1) mma_commit<1>(dfull);
          if (++s == kStages) { s = 0; phase ^= 1; }
        }
        dphase ^= 1;
      }
    }
  } else if (warp < kEpilogueWarp) {
    // ---- rows of no expert
    if (p.zero_free)
      zero_free_rows(p.out, p.out_stride, static_cast<int64_t>(p.n_out) * 2, p.offsets, p.counts, p.E, p.R, blockIdx.x * 2 + warp - 2, gridDim.x * 2);
  } else if (warp < kScaleWarp) {
    // ---- finished accumulators
    const int quarter = warp - kEpilogueWarp;
    uint32_t dphase = 0;
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile x = tile_at<Gated>(p, first, t);
      const int r = quarter * 32 + lane;
      const bool live = r < x.left;
      uint8_t* out = p.out + (static_cast<int64_t>(x.row0) + r) * p.out_stride;
      const float alpha = p.alpha == nullptr ? 1.0f : p.alpha[x.e];
      if (!__all_sync(0xffffffffu, wait_phase(dfull, dphase, give_up, timeouts))) break;
      tmem_fence_after();
      const uint32_t d = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      constexpr int kCols = Gated ? kTileN / 2 : kTileN;
#pragma unroll 1
      for (int c = 0; c < kCols; c += 32) {
        uint32_t v[32], u[32];
        tmem_load32(d + c, v);
        if constexpr (Gated) tmem_load32(d + kTileN / 2 + c, u);
        tmem_wait_load();
        if (live) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            const int n = x.n0 + c + i;
            if (n < p.n_out) {
              float y[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                y[j] = __uint_as_float(v[i + j]) * alpha;
                if constexpr (Gated) y[j] = swiglu(y[j], __uint_as_float(u[i + j]) * alpha);
              }
              *reinterpret_cast<uint4*>(out + static_cast<int64_t>(n) * 2) =
                  make_uint4(Act<T>::pack(y[0], y[1]), Act<T>::pack(y[2], y[3]), Act<T>::pack(y[4], y[5]), Act<T>::pack(y[6], y[7]));
            }
          }
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dempty);
      dphase ^= 1;
    }
  } else {
    // ---- the rows' scales: row r of the tile, chunk i of 64 values, to the word r / 32 of line r % 32 of block i
    uint32_t at = 0;  // stages so far; this warp takes every fourth
    bool ok = true;
    for (uint32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile x = tile_at<Gated>(p, first, t);
      for (int k = 0; k < steps; ++k, ++at) {
        if ((at & 3) != static_cast<uint32_t>(warp - kScaleWarp)) continue;
        const int n = chunks - 4 * k < 4 ? chunks - 4 * k : 4;
        uint32_t w[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = q * 32 + lane;
          const uint8_t* src = p.sf + (static_cast<int64_t>(x.row0) + r) * (p.n_in / 16) + k * 16;
#pragma unroll
          for (int i = 0; i < 4; ++i) w[q][i] = r < x.left && i < n ? __ldg(reinterpret_cast<const uint32_t*>(src) + i) : 0;
        }
        const uint32_t s = at % kStages, phase = at / kStages & 1;
        if (!(ok = __all_sync(0xffffffffu, wait_phase(empty0 + 8 * s, phase ^ 1, give_up, timeouts)))) break;
        const uint32_t sfa = stage0 + s * kStage + kABytes + kBBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sfa + i * 512 + lane * 16), "r"(w[0][i]), "r"(w[1][i]), "r"(w[2][i]), "r"(w[3][i])
                       : "memory");
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(full0 + 8 * s);
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 2) {
    tmem_fence_after();
    tmem_free<1>(tmem, 512);
  }
}

template <bool Gated, typename T>
cudaError_t launch(const Params& p, int64_t most_tiles, bool pdl, cudaStream_t stream) {
  constexpr auto kern = expert_nvfp4_kernel<Gated, T>;
  const cudaError_t e = allow_smem<kern>(kSmem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms == 0) return cudaErrorInvalidDevice;
  return launch_pdl(kern, dim3(static_cast<unsigned>(most_tiles < sms ? most_tiles : sms)), kThreads, kSmem, pdl, stream, p);
}

}  // namespace

cudaError_t launch_expert_matmul_nvfp4(const mfr_expert_matmul_nvfp4_args& a, cudaStream_t stream) {
  Params p = {};
  constexpr CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const int64_t line = a.n_in / 2, wide = a.gated ? 2 * a.n_out : a.n_out;
  cudaError_t e = encode_rows(&p.a, type, a.codes, line, a.num_rows, line, 128, kTileM);
  if (e == cudaSuccess) e = encode_rows(&p.a_small, type, a.codes, line, a.num_rows, line, 128, kSmallRows);
  if (e == cudaSuccess) e = encode_weights(&p.b, type, a.weight_codes, line, wide, a.E, line, wide * line, 128, a.gated ? kTileN / 2 : kTileN);
  if (e != cudaSuccess) return e;
  p.offsets = a.expert_offsets;
  p.counts = a.expert_counts;
  p.sf = static_cast<const uint8_t*>(a.sf);
  p.weight_sf = static_cast<const uint8_t*>(a.weight_sf);
  p.alpha = a.alpha;
  p.E = a.E;
  p.R = static_cast<int32_t>(a.num_rows);
  p.n_in = a.n_in;
  p.n_out = a.n_out;
  p.tiles_n = a.gated ? a.n_out / (kTileN / 2) : (a.n_out + kTileN - 1) / kTileN;
  p.sf_tiles = static_cast<int32_t>((wide + 127) / 128);
  p.zero_free = (a.flags & MFR_FLAG_ZERO_PADDING) != 0;
  p.out = static_cast<uint8_t*>(a.out);
  p.out_stride = a.out_stride * 2;
  const int64_t tiles = expert_row_tiles(a.num_rows, a.E, kTileM) * p.tiles_n;
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0, bf16 = a.out_dtype == MFR_BF16;
  if (a.gated) return bf16 ? launch<true, __nv_bfloat16>(p, tiles, pdl, stream) : launch<true, __half>(p, tiles, pdl, stream);
  return bf16 ? launch<false, __nv_bfloat16>(p, tiles, pdl, stream) : launch<false, __half>(p, tiles, pdl, stream);
}

cudaError_t read_and_reset_expert_nvfp4_timeouts(unsigned int* count) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_expert_nvfp4_wait_timeouts, sizeof(unsigned int));
  if (e != cudaSuccess || *count == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_expert_nvfp4_wait_timeouts, &zero, sizeof(unsigned int));
}

}  // namespace mfr
