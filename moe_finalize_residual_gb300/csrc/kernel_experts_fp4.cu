// The experts' NVFP4 product: rows in expert order times their experts' weights, both as E2M1 codes with an E4M3 scale for
// every 16 values, on the fifth-generation tensor cores, which take codes and scales as they are.
//
// The kernel is that of the 16-bit products (kernel_experts.cu): weight rows in the lanes of tensor memory, an expert's rows
// as its columns, persistent CTAs or pairs of them, operands by tensor copies, results through shared memory.  A stage is 256
// values of the reduction.  The scales take a second way: tensor memory wants them in blocks of 128 rows x 4 scales, which
// the issuing thread copies there from shared memory before each stage's instructions.  The weights' lie in such tiles and
// come by tensor copies as they are; gated, where a tile's lanes are 8 gates and 8 others alternately, six warps, a stage each
// in turn, put them in order.  The rows' scales are row-major, since rows begin anywhere.  With few rows the same warps gather
// them; with many that took longer than the instructions (32 sectors a load; 105 us where 84 go without it), so a kernel
// before this one writes them in tiles, once for all columns' tiles.
//
// What bounds it, on GB300: with few rows HBM (16 tokens of 256 experts, top-8, 7168 x 2048 weights: 123.5 us, the floor); with many
// the stages, 0.35 us each (8 experts of 768 rows, 7168 x 4096: 78 us, 4.6 PFLOP/s): their copies, 34816 bytes a CTA, take most of that
// at the 60 bytes a cycle that come from L2, the instructions 384 cycles; gated the weights' scales on top of it (99 us).
#include "experts_device.cuh"

namespace mfr {

__device__ unsigned int g_expert_nvfp4_wait_timeouts = 0;

namespace {

constexpr int kEpilogueWarp = 4;  // first of kOutGroups groups of four
constexpr int kScaleWarp = kEpilogueWarp + 4 * kOutGroups;
constexpr int kScaleWarps = 6;
constexpr int kThreads = 32 * (kScaleWarp + kScaleWarps);
constexpr int kDepth = 256;       // reduction values of a stage: lines of 128 bytes
constexpr int kTileM = kExpertTileRows;
constexpr int kABytes = kTileM * 128;
constexpr int kSfaBytes = kTileM * kDepth / 16;
constexpr int kBoxRows = 32;      // rows of a box of B
constexpr int kBarBytes = 512;

struct Params {
  CUtensorMap a, b, b_small, sfa, sfb;  // (sfa: not gated; sfb: rows' scales in order; both 512 bytes a row)
  const int32_t* offsets;
  const int32_t* counts;
  const uint8_t* sf;         // rows' scales, row-major
  const uint8_t* weight_sf;  // weights' scales in tiles
  const float* alpha;
  int32_t E, R;
  int32_t n_in, n_out;
  int32_t tiles_m;
  int32_t row_tiles;         // tiles of the rows, at most
  int32_t sf_tiles;          // tiles of 128 weight rows an expert
  int32_t zero_free;
  int32_t test_extra;        // as in kernel_experts.cu
  RowsOut to;
};

template <bool Gated, int Ctas, int BN>
struct Shape {
  static constexpr int kBRows = BN / Ctas;  // rows whose codes this CTA copies (their scales: all BN)
  static constexpr int kBBytes = kBRows * 128;
  static constexpr bool kInOrder = Ctas == 2;         // the rows' scales are, in the workspace
  static constexpr bool kGather = Gated || !kInOrder; // there are scales for the warps to put in order
  static constexpr int kSfBlocks = (BN + 127) / 128;  // blocks of 128 rows' scales
  static constexpr int kSfbBytes = kSfBlocks * 128 * kDepth / 16;
  static constexpr int kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr int kStage = (kStageBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = 209920 / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + kOutGroups * kOutBytes + kBarBytes + (MFR_MAX_EXPERTS + 1 + 32) * 4;
  static constexpr int kFeatures = (Gated ? kTileM / 2 : kTileM) * Ctas;  // values of an output row in a tile
  static constexpr int kUnit = Ctas == 1 ? 16 : 32;
  // tensor-memory columns: two accumulators, then areas of a stage's scales, 4 bytes a lane and column
  static constexpr uint32_t kSfColumns = (kSfaBytes + kSfbBytes) / 128;
  static constexpr int kAreas = 2;
  static_assert(2 * BN + kAreas * kSfColumns <= 512 && kStageBytes % 512 == 0 && kBBytes % 1024 == 0, "tensor memory, alignment");
  static_assert(kSmem <= 232448, "shared memory");
  // (a warp that waits for its stage's place has filled the stage kScaleWarps before; were they more than the places, that
  // place could be two turns behind, which its parity does not show)
  static_assert(kScaleWarps <= kStages, "scale warps");
};

struct Tile {
  int e, row0, rows, m0;
};

template <bool Gated, int Ctas, int BN>
__device__ __forceinline__ Tile tile_at(const Params& p, const int* first, uint32_t t) {
  using S = Shape<Gated, Ctas, BN>;
  Tile x;
  const int m = t / p.tiles_m;
  x.m0 = t % p.tiles_m * S::kFeatures;
  const RowPart part = row_part(first, p.offsets, p.counts, p.E, p.R, m, BN, S::kUnit);
  x.e = part.e;
  x.row0 = part.row0;
  x.rows = part.rows;
  x.e = uniform(x.e);  // (called by whole warps)
  x.row0 = uniform(x.row0);
  x.rows = uniform(x.rows);
  return x;
}

__device__ __forceinline__ void sts128(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <bool Gated, int Ctas, int BN, typename T>
__global__ void __launch_bounds__(kThreads, 1) expert_nvfp4_kernel(const __grid_constant__ Params p) {
  using S = Shape<Gated, Ctas, BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  const uint32_t stage0 = smem_addr(smem);
  uint8_t* boxes = smem + S::kStages * S::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(boxes + kOutGroups * kOutBytes);
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * S::kStages, sf0 = empty0 + 8 * S::kStages;
  const uint32_t dfull0 = sf0 + 8 * S::kStages, dempty0 = dfull0 + 16;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bars + 3 * S::kStages + 4);
  volatile int* give_up = reinterpret_cast<volatile int*>(tmem_at + 1);
  int* first = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);
  static_assert((3 * S::kStages + 5) * 8 <= kBarBytes, "barriers");
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = Ctas == 2 ? uniform(cluster_ctarank()) : 0;
  unsigned int* const timeouts = &g_expert_nvfp4_wait_timeouts;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1 + p.test_extra);  // the copies' bytes
      mbar_init(sf0 + 8 * s, Ctas);   // the scales that the warps put in order
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(dfull0 + 8 * i, 1);
      mbar_init(dempty0 + 8 * i, 4 * kOutGroups * Ctas);
    }
    *give_up = 0;
    fence_mbar_init();
    tma_prefetch_map(&p.a);
    tma_prefetch_map(&p.b);
  }
  if (warp == 2) tmem_alloc<Ctas>(smem_addr(tmem_at), 512);
  pdl_launch_dependents();
  pdl_wait();
  count_tiles(first, first + MFR_MAX_EXPERTS + 1, p.offsets, p.counts, p.E, p.R, BN, p.row_tiles);
  tmem_fence_before();
  if constexpr (Ctas == 2) cluster_sync(); else __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = uniform(*tmem_at);
  const uint32_t tiles = uniform(static_cast<uint32_t>(first[p.E]) * p.tiles_m);
  const uint32_t t0 = blockIdx.x / Ctas, dt = gridDim.x / Ctas;
  const int chunks = p.n_in / 64;  // instructions a tile, and columns of 512 bytes of the scales' tiles

  if (warp == 0) {
    // ---- copies
    uint32_t s = 0, phase = 0;
    bool ok = true;
    for (uint32_t t = t0; t < tiles && ok; t += dt) {
      const Tile x = tile_at<Gated, Ctas, BN>(p, first, t);
      if (x.rows <= 0) continue;
      const int mine = (x.rows + S::kUnit - 1) / S::kUnit * S::kUnit / Ctas;
      const bool whole = S::kBRows <= kBoxRows || mine > S::kBRows / 2;
      const int nboxes = whole ? 1 : (mine + kBoxRows - 1) / kBoxRows;
      const int sf_tile = x.m0 / 128 + rank;  // (not gated) of this CTA's lanes; behind the weights' last row there is none
      const bool sfa = !Gated && sf_tile < p.sf_tiles;
      const int sf_row = (x.e * p.sf_tiles + sf_tile) * chunks;
      const uint32_t codes = kABytes + (whole ? S::kBBytes : nboxes * kBoxRows * 128);
      const int sf_all = Gated ? 0 : Ctas == 2 && x.m0 / 128 + 1 < p.sf_tiles ? 2 : 1;  // of both CTAs
      for (int k = 0; k < chunks; k += 4) {
        if (!(ok = __all_sync(0xffffffffu, wait_phase<Ctas>(empty0 + 8 * s, phase ^ 1, give_up, timeouts)))) break;
        const uint32_t a = stage0 + s * S::kStage, b = a + kABytes;
        if (elect_one()) {
          uint32_t bar = full0 + 8 * s;
          if (rank == 0) mbar_arrive_expect_tx(bar, Ctas * (codes + (S::kInOrder ? S::kSfbBytes : 0)) + sf_all * kSfaBytes);
          if constexpr (Ctas == 2) bar = cluster_addr(bar, 0);
          if constexpr (Gated)
            tma_load_5d<Ctas>(a, &p.a, k * 32, 0, 0, (x.m0 + rank * (kTileM / 2)) / 8, x.e, bar);
          else
            tma_load_3d<Ctas>(a, &p.a, k * 32, x.m0 + rank * kTileM, x.e, bar);
          if (S::kBRows <= kBoxRows || whole) {  // (p.b_small is there for larger tiles alone)
            tma_load_2d<Ctas>(b, &p.b, k * 32, x.row0 + rank * mine, bar);
          } else {
            for (int i = 0; i < nboxes; ++i)
              tma_load_2d<Ctas>(b + i * kBoxRows * 128, &p.b_small, k * 32, x.row0 + rank * mine + i * kBoxRows, bar);
          }
          if (sfa) tma_load_2d<Ctas>(b + S::kBBytes, &p.sfa, 0, sf_row + k, bar);  // (may reach into the next tile's columns)
          if constexpr (S::kInOrder)
            tma_load_2d<Ctas>(b + S::kBBytes + kSfaBytes, &p.sfb, 0, (static_cast<int>(t / p.tiles_m) * chunks + k) * S::kSfBlocks, bar);
        }
        __syncwarp();
        if (++s == S::kStages) { s = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    // ---- matrix instructions (of a pair: by its first CTA)
    if (rank == 0) {
      uint32_t s = 0, phase = 0, buf = 0, dphase = 0, area = 0;
      bool ok = true;
      for (uint32_t t = t0; t < tiles && ok; t += dt) {
        const Tile x = tile_at<Gated, Ctas, BN>(p, first, t);
        if (x.rows <= 0) continue;
        const uint32_t idesc = nvfp4_idesc(kTileM * Ctas, (x.rows + S::kUnit - 1) / S::kUnit * S::kUnit);
        if (!(ok = __all_sync(0xffffffffu, wait_phase<Ctas>(dempty0 + 8 * buf, dphase ^ 1, give_up, timeouts)))) break;
        for (int k = 0; k < chunks; k += 4) {
          if (!(ok = __all_sync(0xffffffffu, wait_phase<1>(full0 + 8 * s, phase, give_up, timeouts) &&
                                                 (!S::kGather || wait_phase<Ctas>(sf0 + 8 * s, phase, give_up, timeouts))))) break;
          tmem_fence_after();
          if (elect_one()) {
            const uint32_t a = stage0 + s * S::kStage, b = a + kABytes, sfa = b + S::kBBytes, sfb = sfa + kSfaBytes;
            const uint64_t da = swizzled_desc(a, 1024, 16), db = swizzled_desc(b, 1024, 16);
            const uint32_t ta = tmem + 2 * BN + area * S::kSfColumns, tb = ta + kSfaBytes / 128;
            const int n = chunks - k < 4 ? chunks - k : 4;
            // (copies and instructions of one thread run in the order of their issue; two areas let the next stage's copies
            // go beside this stage's instructions)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i >= n) break;
              tmem_copy_scales<Ctas>(ta + 4 * i, sfa + 512 * i);
#pragma unroll
              for (int j = 0; j < S::kSfBlocks; ++j) tmem_copy_scales<Ctas>(tb + 4 * (S::kSfBlocks * i + j), sfb + 512 * (S::kSfBlocks * i + j));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i >= n) break;
              mma_nvfp4<Ctas>(tmem + buf * BN, da + 2 * i, db + 2 * i, idesc, ta + 4 * i, tb + 4 * S::kSfBlocks * i, (k | i) != 0);
            }
            mma_commit<Ctas>(empty0 + 8 * s);
            if (k + 4 >= chunks) mma_commit<Ctas>(dfull0 + 8 * buf);
          }
          __syncwarp();
          if (++area == S::kAreas) area = 0;
          if (++s == S::kStages) { s = 0; phase ^= 1; }
        }
        if (buf ^= 1; buf == 0) dphase ^= 1;
      }
    }
  } else if (warp < kEpilogueWarp) {
    // ---- rows of no expert
    if (p.zero_free)
      zero_free_rows(p.to.out, p.to.out_stride, static_cast<int64_t>(p.n_out) * 2, p.offsets, p.counts, p.E, p.R, blockIdx.x * 2 + warp - 2, gridDim.x * 2);
  } else if (warp < kScaleWarp) {
    // ---- finished accumulators
    const int quarter = warp % 4, group = (warp - kEpilogueWarp) / 4;
    uint32_t buf = 0, dphase = 0;
    for (uint32_t t = t0; t < tiles; t += dt) {
      const Tile x = tile_at<Gated, Ctas, BN>(p, first, t);
      if (x.rows <= 0) continue;
      const float alpha = p.alpha == nullptr ? 1.0f : p.alpha[x.e];
      if (!named_all(1 + group, 128, wait_phase<Ctas>(dfull0 + 8 * buf, dphase, give_up, timeouts))) break;  // (the four warps share their stores)
      tmem_fence_after();
      store_tile<T, Gated>(tmem + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16), x.rows, x.row0, x.m0 + rank * (S::kFeatures / Ctas), alpha,
                           p.to, boxes + group * kOutBytes, group);
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (Ctas == 2) mbar_arrive_cluster(cluster_addr(dempty0 + 8 * buf, 0)); else mbar_arrive(dempty0 + 8 * buf);
      }
      if (buf ^= 1; buf == 0) dphase ^= 1;
    }
  } else if constexpr (S::kGather) {
    // ---- scales to put in order: row r of a block, chunk i of 64 values, to word r / 32 of line r % 32 of the chunk's 512
    // bytes.  A warp takes every sixth stage.  It loads the next one's scales as soon as this one's are stored: not before, since
    // the release that says so would wait for the loads.
    const bool wide = p.n_in % 256 == 0 && reinterpret_cast<uintptr_t>(p.sf) % 16 == 0;  // (a row's 16 scales of a stage on 16 bytes)
    const int line = p.n_in / 16;
    uint32_t t = t0, stage = warp - kScaleWarp;
    int k = 4 * static_cast<int>(stage);
    for (bool ok = true;; stage += kScaleWarps, k += 4 * kScaleWarps) {
      // the tile of the stage: over tiles that end before it
      Tile x;
      bool more = false;
      for (; t < tiles; t += dt) {
        x = tile_at<Gated, Ctas, BN>(p, first, t);
        const int all = x.rows > 0 ? (chunks + 3) / 4 * 4 : 0;
        if ((more = k < all)) break;
        k -= all;
      }
      if (!more || !ok) break;
      const int n = chunks - k < 4 ? chunks - k : 4;
      uint32_t w[4];
      if constexpr (!S::kInOrder) {  // at most 32 rows: the first word of each line
        static_assert(S::kInOrder || BN == 32, "one row a lane");
        const uint8_t* src = p.sf + (static_cast<int64_t>(x.row0) + lane) * line + k * 4;
        if (wide) {
          const uint4 v = lane < x.rows ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
          w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = lane < x.rows && i < n ? __ldg(reinterpret_cast<const uint32_t*>(src) + i) : 0;
        }
      }
      uint2 g[4], h[4];
      if constexpr (Gated) {
        // lane l of the block's lines is 8 gates, 8 others and so on: its words are the weights' rows c, c + 16, c + 32 and
        // c + 48 from f0 on, which lie in the lines c and c + 16 of a tile, two neighbouring words each
        const int f0 = x.m0 + rank * (kTileM / 2), f = f0 + (lane & 8 ? p.n_out : 0), c = lane / 16 * 8 + lane % 8;
        const uint8_t* wsf = p.weight_sf + ((static_cast<int64_t>(x.e) * p.sf_tiles + f / 128) * chunks + k) * 512 + c * 16 + f0 % 128 / 32 * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = i < n ? __ldg(reinterpret_cast<const uint2*>(wsf + i * 512)) : make_uint2(0, 0);
          h[i] = i < n ? __ldg(reinterpret_cast<const uint2*>(wsf + i * 512 + 256)) : make_uint2(0, 0);
        }
      }
      const uint32_t s = stage % S::kStages, phase = stage / S::kStages & 1;
      if (!(ok = __all_sync(0xffffffffu, wait_phase<Ctas>(empty0 + 8 * s, phase ^ 1, give_up, timeouts)))) break;
      const uint32_t sfa = stage0 + s * S::kStage + kABytes + S::kBBytes + lane * 16, sfb = sfa + kSfaBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (!S::kInOrder) sts128(sfb + i * 512, w[i], 0, 0, 0);
        if constexpr (Gated) sts128(sfa + i * 512, g[i].x, h[i].x, g[i].y, h[i].y);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        if constexpr (Ctas == 2) mbar_arrive_cluster(cluster_addr(sf0 + 8 * s, 0)); else mbar_arrive(sf0 + 8 * s);
      }
    }
  }
  if (warp < 2) drain(give_up);
  __syncwarp();
  tmem_fence_before();
  if constexpr (Ctas == 2) cluster_sync(); else __syncthreads();
  if (warp == 2) {
    tmem_fence_after();
    tmem_free<Ctas>(tmem, 512);
  }
}

// The rows' scales in the order of tensor memory: for each tile of kNvfp4Rows rows and each chunk of 64 values two blocks of 128
// rows, row r's four scales in word r / 32 of line r % 32 of 16 bytes.  A CTA takes 16 chunks of a tile at a time, through shared
// memory: rows in 64-byte pieces on one side, whole blocks on the other.  Rows of no tile get zeros.
constexpr int kOrderThreads = 256, kOrderChunks = 16, kOrderRows = 256, kOrderPitch = kOrderChunks + 1;
struct OrderParams {
  const uint8_t* sf;
  const int32_t* offsets;
  const int32_t* counts;
  int32_t E, R, chunks;
  int32_t tiles;  // of the rows, at most: the workspace holds so many
  uint8_t* to;
};
__global__ void __launch_bounds__(kOrderThreads) order_scales_kernel(const __grid_constant__ OrderParams p) {
  static_assert(kNvfp4Rows > 128 && kNvfp4Rows <= kOrderRows, "two blocks of rows");
  __shared__ uint32_t words[kOrderRows * kOrderPitch];
  __shared__ int first[MFR_MAX_EXPERTS + 1 + 32];
  pdl_launch_dependents();
  pdl_wait();
  count_tiles(first, first + MFR_MAX_EXPERTS + 1, p.offsets, p.counts, p.E, p.R, kNvfp4Rows, p.tiles);
  const int groups = (p.chunks + kOrderChunks - 1) / kOrderChunks;
  const int64_t all = static_cast<int64_t>(first[p.E]) * groups;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    const int m = static_cast<int>(i / groups), c0 = static_cast<int>(i % groups) * kOrderChunks;
    const RowPart x = row_part(first, p.offsets, p.counts, p.E, p.R, m, kNvfp4Rows, 32);
    const int n = p.chunks - c0 < kOrderChunks ? p.chunks - c0 : kOrderChunks;
    __syncthreads();  // (the last turn's words are read)
#pragma unroll 4
    for (int at = threadIdx.x; at < kOrderRows * kOrderChunks; at += kOrderThreads) {
      const int r = at / kOrderChunks, c = at % kOrderChunks;
      words[r * kOrderPitch + c] =
          r < x.rows && c < n ? __ldg(reinterpret_cast<const uint32_t*>(p.sf + ((static_cast<int64_t>(x.row0) + r) * p.chunks + c0 + c) * 4)) : 0;
    }
    __syncthreads();
    for (int at = threadIdx.x; at < n * 64; at += kOrderThreads) {
      const int c = at / 64, b = at / 32 % 2, l = at % 32;
      const uint32_t* w = words + (b * 128 + l) * kOrderPitch + c;
      *reinterpret_cast<uint4*>(p.to + (((static_cast<int64_t>(m) * p.chunks + c0 + c) * 2 + b) * 32 + l) * 16) =
          make_uint4(w[0], w[32 * kOrderPitch], w[64 * kOrderPitch], w[96 * kOrderPitch]);
    }
  }
}

template <bool Gated, int Ctas, int BN, typename T>
cudaError_t launch(const Params& p, int64_t tiles, bool pdl, cudaStream_t stream) {
  using S = Shape<Gated, Ctas, BN>;
  constexpr auto kern = expert_nvfp4_kernel<Gated, Ctas, BN, T>;
  const cudaError_t e = allow_smem<kern>(S::kSmem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count() / Ctas * Ctas;
  if (sms == 0) return cudaErrorInvalidDevice;
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles * Ctas < sms ? tiles * Ctas : sms)), kThreads, S::kSmem, pdl, stream, p, Ctas);
}

template <bool Gated, int Ctas, int BN>
cudaError_t launch_tile(const mfr_expert_matmul_nvfp4_args& a, Params& p, cudaStream_t stream) {
  using S = Shape<Gated, Ctas, BN>;
  constexpr CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const int64_t line = a.n_in / 2;
  cudaError_t e = encode_rows(&p.b, type, a.codes, line, a.num_rows, line, 128, S::kBRows);
  if (e == cudaSuccess && S::kBRows > kBoxRows) e = encode_rows(&p.b_small, type, a.codes, line, a.num_rows, line, 128, kBoxRows);
  if (e != cudaSuccess) return e;
  p.tiles_m = (a.n_out + S::kFeatures - 1) / S::kFeatures;
  p.row_tiles = static_cast<int32_t>(expert_row_tiles(a.num_rows, a.E, BN));
  const int64_t tiles = static_cast<int64_t>(p.row_tiles) * p.tiles_m;
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  return a.out_dtype == MFR_BF16 ? launch<Gated, Ctas, BN, __nv_bfloat16>(p, tiles, pdl, stream) : launch<Gated, Ctas, BN, __half>(p, tiles, pdl, stream);
}

// The tile by the rows that an expert has, as in kernel_experts.cu.
template <bool Gated>
cudaError_t launch_by_rows(const mfr_expert_matmul_nvfp4_args& a, Params& p, cudaStream_t stream) {
  if (nvfp4_few_rows(a.num_rows, a.E)) return launch_tile<Gated, 1, 32>(a, p, stream);
  const int chunks = a.n_in / 64;
  const int64_t blocks = expert_row_tiles(a.num_rows, a.E, kNvfp4Rows) * chunks * 2;
  const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(blocks)}, strides[1] = {512};
  const cuuint32_t box[2] = {128, 8};
  cudaError_t e = encode_map(&p.sfb, CU_TENSOR_MAP_DATA_TYPE_INT32, a.workspace, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e != cudaSuccess) return e;
  const OrderParams o = {p.sf, p.offsets, p.counts, p.E, p.R, chunks, static_cast<int32_t>(blocks / 2 / chunks), static_cast<uint8_t*>(a.workspace)};
  const int64_t turns = blocks / 2 / chunks * ((chunks + kOrderChunks - 1) / kOrderChunks), most = int64_t{sm_count()} * 4;
  e = launch_pdl(order_scales_kernel, dim3(static_cast<unsigned>(turns < most ? turns : most)), kOrderThreads, 0, (a.flags & MFR_FLAG_PDL) != 0, stream, o);
  return e != cudaSuccess ? e : launch_tile<Gated, 2, kNvfp4Rows>(a, p, stream);
}

}  // namespace

cudaError_t launch_expert_matmul_nvfp4(const mfr_expert_matmul_nvfp4_args& a, cudaStream_t stream) {
  Params p = {};
  constexpr CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const int64_t line = a.n_in / 2, wide = a.gated ? int64_t{2} * a.n_out : a.n_out;
  const cudaError_t e = a.gated ? encode_gated_weights(&p.a, type, a.weight_codes, line, a.n_out, a.E, line, wide * line, 128)
                                : encode_weights(&p.a, type, a.weight_codes, line, a.n_out, a.E, line, wide * line, 128, kTileM);
  if (e != cudaSuccess) return e;
  p.sf_tiles = static_cast<int32_t>((wide + 127) / 128);
  if (!a.gated) {
    const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(a.E) * p.sf_tiles * (a.n_in / 64)}, strides[1] = {512};
    const cuuint32_t box[2] = {128, 4};
    const cudaError_t es = encode_map(&p.sfa, CU_TENSOR_MAP_DATA_TYPE_INT32, a.weight_sf, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (es != cudaSuccess) return es;
  }
  p.offsets = a.expert_offsets;
  p.counts = a.expert_counts;
  p.sf = static_cast<const uint8_t*>(a.sf);
  p.weight_sf = static_cast<const uint8_t*>(a.weight_sf);
  p.alpha = a.alpha;
  p.E = a.E;
  p.R = static_cast<int32_t>(a.num_rows);
  p.n_in = a.n_in;
  p.n_out = a.n_out;
  p.zero_free = (a.flags & MFR_FLAG_ZERO_PADDING) != 0;
  p.test_extra = (a.flags & MFR_FLAG_TEST_STREAM_TIMEOUT) != 0;
  p.to = {static_cast<uint8_t*>(a.out), a.out_stride * 2, nullptr, 0, a.n_out};
  return a.gated ? launch_by_rows<true>(a, p, stream) : launch_by_rows<false>(a, p, stream);
}

cudaError_t read_expert_nvfp4_timeouts(unsigned int* count) { return cudaMemcpyFromSymbol(count, g_expert_nvfp4_wait_timeouts, sizeof(unsigned int)); }

}  // namespace mfr
