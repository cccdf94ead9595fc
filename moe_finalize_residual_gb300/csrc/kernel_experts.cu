// The experts' 16-bit products: rows in expert order times their experts' weights, and the gradients to the rows and to
// the weights, on the fifth-generation tensor cores.
//
// The three directions are one kernel over tiles of D = A * B summed over the reduction, D's rows in the lanes of tensor
// memory and its columns in tensor memory's:
//   forward          A = weight [n, i]        B = rows [r, i]         over i: both operands' lines run along the reduction
//   gradient to rows A = weight [n, i]        B = d_out [r, n]        over n: A's lines run along D's rows i
//   to weights       A = d_out [r, n]         B = rows [r, i]         over the expert's rows r: both along D's rows and columns
// The instruction takes either kind of lines, so nothing is transposed in memory.  An expert's rows are D's columns in the
// first two: an instruction takes any multiple of 16 (a pair's: 32) of them, so a ragged expert costs what its rows cost,
// and a decode step's few rows hardly anything beside the weights.
//
// A persistent CTA, or a pair of CTAs that share the columns' operand, takes tiles of 128 (256) weight rows x at most BN
// rows.  One warp copies the operands in by tensor copies, 64 values of the reduction a stage; one thread issues the matrix
// instructions into one of two accumulators in tensor memory; two groups of four warps take finished accumulators out, round and
// store them meanwhile.
//
// What bounds it, on GB300: with few rows HBM (64 tokens of 256 experts, top-8, 1024 x 6144 weights: 375 us, every weight read
// once); with many the tensor pipe, active for 92 % of the time (8 experts of 768 rows, 7168 x 4096: 211 us, 1.70 PFLOP/s; the counter
// counts instructions that wait for operands too), beside copies of 64 bytes a cycle and SM, which alone take 0.8 of that; the weights'
// gradient its results beside those copies (64 experts of 384 rows, 4096 x 4096: 645 us by one CTA a tile; by pairs, as from 512 rows
// on, 720 to 750, of it 530 without stores and 404 without results).
#include "experts_device.cuh"

namespace mfr {

__device__ unsigned int g_expert_wait_timeouts = 0;

namespace {

enum Dir { kForward = 0, kGated = 1, kRowsGrad = 2, kWeightGrad = 3 };

constexpr int kEpilogueWarp = 4;                 // first of kOutGroups groups of four
constexpr int kThreads = 32 * (kEpilogueWarp + 4 * kOutGroups);
constexpr int kDepth = 64;                       // reduction values of a stage: lines of 128 bytes
constexpr int kTileM = kExpertTileRows;          // rows of A of one CTA
constexpr int kABytes = kTileM * kDepth * 2;
constexpr int kBoxRows = 32;                     // rows of a small box of B
constexpr int kBarBytes = 512;

struct Params {
  CUtensorMap a, b, b_small, d;  // (d: the weights' gradient)
  const int32_t* offsets;
  const int32_t* counts;
  int32_t E, R;
  int32_t n_red;       // reduction length (the weights' gradient: the expert's rows)
  int32_t n_m;         // values of an output row, as in `to` (the weights' gradient: rows of D)
  int32_t n_n;         // the weights' gradient: columns of D
  int32_t tiles_m, tiles_n;  // row tiles of D; the weights' gradient: column tiles
  int32_t row_tiles;   // tiles of the rows in expert order, at most (but for the weights' gradient)
  int32_t zero_free, accumulate;
  int32_t test_extra;  // arrivals that a stage's barrier expects and that never come (1 only under the failure-detection test hook)
  RowsOut to;          // (but for the weights' gradient)
};

template <int D, int Ctas, int BN>
struct Shape {
  static constexpr int kBRows = BN / Ctas;  // columns of D whose operand this CTA copies
  static constexpr int kBBytes = kBRows * kDepth * 2;
  static constexpr int kStage = kABytes + kBBytes;
  // results leave by a buffer for each group of warps: 128 lines of 128 bytes of the weights' gradient, or 32 rows of the tile's values
  static constexpr int kOut = D == kWeightGrad ? kTileM * 128 : kOutBytes;
  static constexpr int kStages = D == kWeightGrad ? 196608 / kStage : 204800 / kStage;
  static constexpr bool kALines = D == kRowsGrad || D == kWeightGrad;
  static constexpr bool kBLines = D == kWeightGrad;
  static constexpr int kFeatures = (D == kGated ? kTileM / 2 : kTileM) * Ctas;  // values of an output row in a tile
  static constexpr int kUnit = Ctas == 1 ? 16 : 32;  // an instruction's columns are a multiple
  // what one CTA holds besides the stages: the barriers and, but for the weights' gradient, the experts' first tiles
  static constexpr int kFixed = kBarBytes + (D == kWeightGrad ? 0 : (MFR_MAX_EXPERTS + 1 + 32) * 4);
  static constexpr int kSmem = 1024 + kStages * kStage + kOutGroups * kOut + kFixed;
};

struct Tile {
  int e;      // expert
  int row0;   // its first row in the tile (weights' gradient: its first row)
  int rows;   // its rows in the tile (weights' gradient: its rows)
  int m0;     // first value of the output row (weights' gradient: first row of D)
  int n0;     // weights' gradient: first column of D
  int steps;  // stages of the reduction
};

template <int D, int Ctas, int BN>
__device__ __forceinline__ Tile tile_at(const Params& p, const int* first, uint32_t t) {
  using S = Shape<D, Ctas, BN>;
  Tile x;
  if constexpr (D == kWeightGrad) {
    const uint32_t per = static_cast<uint32_t>(p.tiles_m) * p.tiles_n;
    x.e = t / per;
    const uint32_t in = t % per;
    x.m0 = in / p.tiles_n * S::kFeatures;
    x.n0 = in % p.tiles_n * BN;
    const RowSpan s = expert_rows(p.offsets, p.counts, x.e, p.R);
    x.row0 = s.begin;
    x.rows = s.end - s.begin;
    x.steps = (x.rows + kDepth - 1) / kDepth;
  } else {
    const int m = t / p.tiles_m;
    x.m0 = t % p.tiles_m * S::kFeatures;
    x.n0 = 0;
    const RowPart part = row_part(first, p.offsets, p.counts, p.E, p.R, m, BN, S::kUnit);
    x.e = part.e;
    x.row0 = part.row0;
    x.rows = part.rows;
    x.steps = x.rows > 0 ? (p.n_red + kDepth - 1) / kDepth : 0;
  }
  x.e = uniform(x.e);  // (called by whole warps)
  x.row0 = uniform(x.row0);
  x.rows = uniform(x.rows);
  x.steps = uniform(x.steps);
  return x;
}

// Zeros, by one warp, in the lines from `from` on of a stage whose operands' lines are steps of the reduction: they hold rows
// behind the expert's last, which must not count.  In both operands, since 0 * NaN is NaN.
template <typename S>
__device__ __forceinline__ void clear_lines(uint32_t stage, int from) {
  constexpr int kBlock = 64 * kDepth * 2;  // bytes of 64 columns, line by line
#pragma unroll
  for (int block = 0; block < S::kStage / kBlock; ++block)
    for (int at = from * 128 + (threadIdx.x & 31) * 16; at < kBlock; at += 512)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(stage + block * kBlock + at), "r"(0) : "memory");
  fence_async_shared();
  __syncwarp();
}

// T: the operands' type; O: that of D (FP32 for the weights' gradient alone).
template <int D, int Ctas, int BN, typename T, typename O>
__global__ void __launch_bounds__(kThreads, 1) expert_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, Ctas, BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  const uint32_t stage0 = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kStages * S::kStage + kOutGroups * S::kOut);
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * S::kStages;
  // (the next two kinds: the weights' gradient alone)
  const uint32_t tail0 = empty0 + 8 * S::kStages, ready0 = tail0 + 8 * S::kStages;
  const uint32_t dfull0 = ready0 + 8 * S::kStages, dempty0 = dfull0 + 16;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bars + 4 * S::kStages + 4);
  volatile int* give_up = reinterpret_cast<volatile int*>(tmem_at + 1);
  // stages whose copies this CTA has issued: the weights' gradient alone, whose reductions are as long as an expert has rows
  volatile uint32_t* progress = D == kWeightGrad ? tmem_at + 2 : nullptr;
  int* first = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);
  static_assert((4 * S::kStages + 6) * 8 <= kBarBytes, "barriers");

  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = Ctas == 2 ? uniform(cluster_ctarank()) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1 + p.test_extra);
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(tail0 + 8 * s, 1);
      mbar_init(ready0 + 8 * s, Ctas);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(dfull0 + 8 * i, 1);
      mbar_init(dempty0 + 8 * i, 4 * kOutGroups * Ctas);
    }
    *give_up = 0;
    if constexpr (D == kWeightGrad) *progress = 0;
    fence_mbar_init();
    tma_prefetch_map(&p.a);
    tma_prefetch_map(&p.b);
  }
  if (warp == 2) tmem_alloc<Ctas>(smem_addr(tmem_at), 2 * BN);
  pdl_launch_dependents();
  pdl_wait();
  if constexpr (D != kWeightGrad)
    count_tiles(first, first + MFR_MAX_EXPERTS + 1, p.offsets, p.counts, p.E, p.R, BN, p.row_tiles);
  tmem_fence_before();
  if constexpr (Ctas == 2) cluster_sync(); else __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = uniform(*tmem_at);
  const uint32_t tiles = uniform(D == kWeightGrad ? static_cast<uint32_t>(p.E) * p.tiles_m * p.tiles_n : static_cast<uint32_t>(first[p.E]) * p.tiles_m);
  const uint32_t t0 = blockIdx.x / Ctas, dt = gridDim.x / Ctas;

  if (warp == 0) {
    // ---- copies
    uint32_t s = 0, phase = 0;
    bool ok = true;
    for (uint32_t t = t0; t < tiles && ok; t += dt) {
      const Tile x = tile_at<D, Ctas, BN>(p, first, t);
      // B's boxes may reach behind the expert's last row: that only makes columns of D that are not stored
      const int mine = (x.rows + S::kUnit - 1) / S::kUnit * S::kUnit / Ctas;  // rows that this CTA copies, but for the boxes' ends
      const bool whole = S::kBRows <= kBoxRows || mine > S::kBRows / 2;  // one box for all of them, or several of 32
      const int boxes = whole ? 1 : (mine + kBoxRows - 1) / kBoxRows;
      const uint32_t bytes = kABytes + (D == kWeightGrad || whole ? S::kBBytes : boxes * kBoxRows * kDepth * 2);
      for (int k = 0; k < x.steps; ++k) {
        if (!(ok = __all_sync(0xffffffffu, wait_phase<Ctas>(empty0 + 8 * s, phase ^ 1, give_up, &g_expert_wait_timeouts)))) break;
        if (elect_one()) {
          uint32_t bar = full0 + 8 * s;
          if (D == kWeightGrad && x.rows < (k + 1) * kDepth) {
            // the expert's last rows: each CTA sees its own copies land, and clears the lines behind them
            if (rank == 0) mbar_arrive(bar);
            bar = tail0 + 8 * s;
            mbar_arrive_expect_tx(bar, bytes);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(bar, Ctas * bytes);
            if constexpr (Ctas == 2) bar = cluster_addr(bar, 0);
          }
          const uint32_t a = stage0 + s * S::kStage, b = a + kABytes;
          const int r0 = k * kDepth;
          if constexpr (D == kWeightGrad) {
            *progress = *progress + 1;
#pragma unroll
            for (int i = 0; i < kTileM / 64; ++i)
              tma_load_2d<Ctas>(a + i * 64 * kDepth * 2, &p.a, x.m0 + rank * kTileM + i * 64, x.row0 + r0, bar);
#pragma unroll
            for (int i = 0; i < S::kBRows / 64; ++i)
              tma_load_2d<Ctas>(b + i * 64 * kDepth * 2, &p.b, x.n0 + rank * S::kBRows + i * 64, x.row0 + r0, bar);
          } else {
            if constexpr (D == kForward) {
              tma_load_3d<Ctas>(a, &p.a, r0, x.m0 + rank * kTileM, x.e, bar);
            } else if constexpr (D == kGated) {  // 8 rows of the gate, 8 of the others, and so on
              tma_load_5d<Ctas>(a, &p.a, r0, 0, 0, (x.m0 + rank * (kTileM / 2)) / 8, x.e, bar);
            } else {
#pragma unroll
              for (int i = 0; i < kTileM / 64; ++i)
                tma_load_3d<Ctas>(a + i * 64 * kDepth * 2, &p.a, x.m0 + rank * kTileM + i * 64, r0, x.e, bar);
            }
            if (S::kBRows <= kBoxRows || whole) {  // (p.b_small is there for larger tiles alone)
              tma_load_2d<Ctas>(b, &p.b, r0, x.row0 + rank * mine, bar);
            } else {
              for (int i = 0; i < boxes; ++i)
                tma_load_2d<Ctas>(b + i * kBoxRows * kDepth * 2, &p.b_small, r0, x.row0 + rank * mine + i * kBoxRows, bar);
            }
          }
        }
        __syncwarp();
        if (++s == S::kStages) { s = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    // ---- matrix instructions (of a pair: by its first CTA)
    uint32_t s = 0, phase = 0, buf = 0, dphase = 0, tail_phase = 0;
    bool ok = rank == 0;
    for (uint32_t t = t0; t < tiles && ok; t += dt) {
      const Tile x = tile_at<D, Ctas, BN>(p, first, t);
      if (x.steps == 0) continue;
      const int columns = D == kWeightGrad ? BN : (x.rows + S::kUnit - 1) / S::kUnit * S::kUnit;
      const uint32_t idesc = f16_idesc(kIsBf16<T>, S::kALines, S::kBLines, kTileM * Ctas, columns);
      if (!(ok = __all_sync(0xffffffffu, wait_phase<Ctas>(dempty0 + 8 * buf, dphase ^ 1, give_up, &g_expert_wait_timeouts)))) break;
      tmem_fence_after();
      for (int k = 0; k < x.steps; ++k) {
        if (!(ok = __all_sync(0xffffffffu, wait_phase<Ctas>(full0 + 8 * s, phase, give_up, &g_expert_wait_timeouts)))) break;
        if constexpr (D == kWeightGrad) {
          if (k + 1 == x.steps && x.rows % kDepth != 0) {
            if (!(ok = __all_sync(0xffffffffu, wait_phase<Ctas>(ready0 + 8 * s, tail_phase >> s & 1, give_up, &g_expert_wait_timeouts)))) break;
            tail_phase ^= 1u << s;
          }
        }
        tmem_fence_after();
        if (elect_one()) {
          const uint32_t a = stage0 + s * S::kStage, b = a + kABytes;
          const uint64_t da = S::kALines ? swizzled_desc(a, 1024, 64 * kDepth * 2) : swizzled_desc(a, 1024, 16);
          const uint64_t db = S::kBLines ? swizzled_desc(b, 1024, 64 * kDepth * 2) : swizzled_desc(b, 1024, 16);
#pragma unroll
          for (int i = 0; i < kDepth / 16; ++i)  // 16 values of the reduction: 32 bytes of a line, or 16 lines
            mma_f16<Ctas>(tmem + buf * BN, da + i * (S::kALines ? 128 : 2), db + i * (S::kBLines ? 128 : 2), idesc, (k | i) != 0);
          mma_commit<Ctas>(empty0 + 8 * s);
          if (k + 1 == x.steps) mma_commit<Ctas>(dfull0 + 8 * buf);
        }
        __syncwarp();
        if (++s == S::kStages) { s = 0; phase ^= 1; }
      }
      if (buf ^= 1; buf == 0) dphase ^= 1;
    }
  } else if (D == kWeightGrad && warp == 2) {
    // ---- lines behind an expert's last row, cleared as soon as they land: stages before the instructions come to them
    uint32_t s = 0, tail_phase = 0;
    for (uint32_t t = t0; t < tiles; t += dt) {
      const Tile x = tile_at<D, Ctas, BN>(p, first, t);
      if (x.steps == 0) continue;
      s = (s + x.steps - 1) % S::kStages;  // the last stage
      if (x.rows % kDepth != 0) {
        if (!__all_sync(0xffffffffu, wait_phase<1>(tail0 + 8 * s, tail_phase >> s & 1, give_up, &g_expert_wait_timeouts, progress))) break;
        tail_phase ^= 1u << s;
        clear_lines<S>(stage0 + s * S::kStage, x.rows % kDepth);
        if (lane == 0) {
          if constexpr (Ctas == 2) mbar_arrive_cluster(cluster_addr(ready0 + 8 * s, 0)); else mbar_arrive(ready0 + 8 * s);
        }
      }
      s = (s + 1) % S::kStages;
    }
  } else if (warp < kEpilogueWarp) {
    // ---- rows of no expert
    if (D != kWeightGrad && p.zero_free) {
      const int w = blockIdx.x * 2 + warp - 2, nw = gridDim.x * 2;
      zero_free_rows(p.to.out, p.to.out_stride, static_cast<int64_t>(p.n_m) * 2, p.offsets, p.counts, p.E, p.R, w, nw);
      if (D == kGated && p.to.gate_up != nullptr)
        zero_free_rows(p.to.gate_up, p.to.gate_up_stride, static_cast<int64_t>(p.n_m) * 4, p.offsets, p.counts, p.E, p.R, w, nw);
    }
  } else {
    // ---- finished accumulators
    const int quarter = warp % 4, group = (warp - kEpilogueWarp) / 4, sync = 1 + group;
    uint32_t buf = 0, dphase = 0;
    for (uint32_t t = t0; t < tiles; t += dt) {
      const Tile x = tile_at<D, Ctas, BN>(p, first, t);
      const bool some = x.steps > 0;
      if (some) {
        const bool ok = wait_phase<Ctas>(dfull0 + 8 * buf, dphase, give_up, &g_expert_wait_timeouts, progress);
        if (!named_all(sync, 128, ok)) break;  // (the four warps share their stores)
        tmem_fence_after();
      }
      const uint32_t d = tmem + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16);
      const int r = quarter * 32 + lane;  // this thread's lane of D
      if constexpr (D == kWeightGrad) {
        // through shared memory, since a thread has a row: lines of 128 bytes (kLine values) of 128 rows, a box each
        constexpr int kLine = 128 / sizeof(O);
        const int m0 = x.m0 + rank * kTileM;
        if (some || !p.accumulate) {
          // (each group half of the columns, by a buffer of its own)
          const uint32_t box = stage0 + S::kStages * S::kStage + group * S::kOut;
          const bool first_thread = threadIdx.x % 128 == 0;
#pragma unroll 1
          for (int c = group * (BN / 2); c < (group + 1) * (BN / 2) && x.n0 + c < p.n_n; c += kLine) {
            uint32_t v[kLine];
            if (some) {
#pragma unroll
              for (int h = 0; h < kLine; h += 32) tmem_load32(d + c + h, v + h);
              tmem_wait_load(v);
              if constexpr (kLine == 64) tmem_after_wait(v + 32);
            } else {
#pragma unroll
              for (int i = 0; i < kLine; ++i) v[i] = 0;
            }
            if (first_thread) tma_store_wait_read<0>();  // the buffer's last box has left it
            named_sync(sync, 128);
            constexpr int kPiece = 16 / sizeof(O);  // values of 16 bytes, in the 128-byte swizzle
#pragma unroll
            for (int i = 0; i < kLine; i += kPiece) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(O) == 4)
                  w[j] = v[i + j];
                else
                  w[j] = Act<T>::pack(__uint_as_float(v[i + 2 * j]), __uint_as_float(v[i + 2 * j + 1]));
              }
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + r * 128 + (((i / kPiece) ^ (r & 7)) << 4)), "r"(w[0]), "r"(w[1]),
                           "r"(w[2]), "r"(w[3])
                           : "memory");
            }
            fence_async_shared();
            named_sync(sync, 128);
            if (first_thread) {
              if (m0 < p.n_m) {
                if (p.accumulate)
                  tma_add_3d(&p.d, box, x.n0 + c, m0, x.e);
                else
                  tma_store_3d(&p.d, box, x.n0 + c, m0, x.e);
              }
              tma_store_commit();
            }
          }
        }
      } else {
        store_tile<T, D == kGated>(d, x.rows, x.row0, x.m0 + rank * (S::kFeatures / Ctas), 1.0f, p.to, smem + S::kStages * S::kStage + group * S::kOut,
                                     group);
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
    if (D == kWeightGrad && threadIdx.x % 128 == 0) tma_store_wait();
  }
  if (warp < 2) drain(give_up);
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
cudaError_t launch_rows(int act, int64_t R, int E, const void* rows, int64_t rows_stride, Params& p, bool pdl, cudaStream_t stream) {
  using S = Shape<D, Ctas, BN>;
  static_assert(S::kBRows % kBoxRows == 0, "boxes of B");
  cudaError_t e = encode_rows(&p.b, map_type(act), rows, p.n_red, R, rows_stride * 2, kDepth, S::kBRows);
  if (e == cudaSuccess && S::kBRows > kBoxRows) e = encode_rows(&p.b_small, map_type(act), rows, p.n_red, R, rows_stride * 2, kDepth, kBoxRows);
  if (e != cudaSuccess) return e;
  p.tiles_m = (p.n_m + S::kFeatures - 1) / S::kFeatures;
  p.row_tiles = static_cast<int32_t>(expert_row_tiles(R, E, BN));
  const int64_t tiles = static_cast<int64_t>(p.row_tiles) * p.tiles_m;
  return act == MFR_BF16 ? launch<D, Ctas, BN, __nv_bfloat16, __nv_bfloat16>(p, tiles, pdl, stream)
                         : launch<D, Ctas, BN, __half, __half>(p, tiles, pdl, stream);
}

// The tile by the rows that an expert has: with few of them the stages hold little but weights, as many as fit; with many, a pair
// of CTAs halves the copies of the columns' operand.  Measured, 64 experts of 4096 x 4096 in BF16 (floor 317 us): 2 rows each
// 310 us by the small tile and 317 by the pair's, 16 rows 319 and 325, 32 rows 324 and 328, 48 rows (two small tiles an expert)
// 379 and 331.  Rows vary from expert to expert, so the border is well below 32.  R is the buffer's rows: those of routes elsewhere
// and of the experts' alignment count too, so a decode step in a buffer aligned to 128 goes by the pair's tile (64 tokens of 256 experts,
// top-8, 1024 x 6144: 377 us by it, 382 by the small one without alignment).
template <int D>
cudaError_t launch_by_rows(int act, int64_t R, int E, const void* rows, int64_t rows_stride, Params& p, bool pdl, cudaStream_t stream) {
  if (R <= int64_t{16} * E) return launch_rows<D, 1, 32>(act, R, E, rows, rows_stride, p, pdl, stream);
  return launch_rows<D, 2, 256>(act, R, E, rows, rows_stride, p, pdl, stream);
}

}  // namespace

cudaError_t launch_expert_matmul(const mfr_expert_matmul_args& a, cudaStream_t stream) {
  Params p = {};
  const CUtensorMapDataType type = map_type(a.act_dtype);
  const int64_t row = a.weight_stride * 2, wide = a.gated ? int64_t{2} * a.n_out : a.n_out;
  const int64_t expert = (a.E > 1 ? a.weight_expert_stride * 2 : wide * row);
  cudaError_t e;
  if (a.gated) {
    e = encode_gated_weights(&p.a, type, a.weight, a.n_in, a.n_out, a.E, row, expert, kDepth);
  } else {
    e = encode_weights(&p.a, type, a.weight, a.n_in, a.n_out, a.E, row, expert, kDepth, kTileM);
  }
  if (e != cudaSuccess) return e;
  p.offsets = a.expert_offsets;
  p.counts = a.expert_counts;
  p.E = a.E;
  p.R = static_cast<int32_t>(a.num_rows);
  p.n_red = a.n_in;
  p.n_m = a.n_out;
  p.zero_free = (a.flags & MFR_FLAG_ZERO_PADDING) != 0;
  p.test_extra = (a.flags & MFR_FLAG_TEST_STREAM_TIMEOUT) != 0;
  p.to = {static_cast<uint8_t*>(a.out), a.out_stride * 2, static_cast<uint8_t*>(a.gate_up), a.gate_up_stride * 2, a.n_out};
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  return a.gated ? launch_by_rows<kGated>(a.act_dtype, a.num_rows, a.E, a.rows, a.rows_stride, p, pdl, stream)
                 : launch_by_rows<kForward>(a.act_dtype, a.num_rows, a.E, a.rows, a.rows_stride, p, pdl, stream);
}

cudaError_t launch_expert_rows_grad(const mfr_expert_matmul_backward_args& a, cudaStream_t stream) {
  Params p = {};
  const cudaError_t e = encode_weights(&p.a, map_type(a.act_dtype), a.weight, a.n_in, a.n_out, a.E, a.weight_stride * 2,
                                       (a.E > 1 ? a.weight_expert_stride : a.n_out * a.weight_stride) * 2, 64, kDepth);
  if (e != cudaSuccess) return e;
  p.offsets = a.expert_offsets;
  p.counts = a.expert_counts;
  p.E = a.E;
  p.R = static_cast<int32_t>(a.num_rows);
  p.n_red = a.n_out;
  p.n_m = a.n_in;
  p.zero_free = (a.flags & MFR_FLAG_ZERO_PADDING) != 0;
  p.test_extra = (a.flags & MFR_FLAG_TEST_STREAM_TIMEOUT) != 0;
  p.to = {static_cast<uint8_t*>(a.d_rows), a.d_rows_stride * 2, nullptr, 0, a.n_in};
  return launch_by_rows<kRowsGrad>(a.act_dtype, a.num_rows, a.E, a.d_out, a.d_out_stride, p, (a.flags & MFR_FLAG_PDL) != 0, stream);
}

namespace {

template <int Ctas>
cudaError_t launch_weights(const mfr_expert_matmul_backward_args& a, Params& p, cudaStream_t stream) {
  constexpr int BN = 256;
  p.tiles_m = (a.n_out + kTileM * Ctas - 1) / (kTileM * Ctas);
  p.tiles_n = (a.n_in + BN - 1) / BN;
  const int64_t tiles = static_cast<int64_t>(a.E) * p.tiles_m * p.tiles_n;
  const bool pdl = (a.flags & MFR_FLAG_PDL) != 0;
  if (a.d_weight_dtype == MFR_FP32)
    return a.act_dtype == MFR_BF16 ? launch<kWeightGrad, Ctas, BN, __nv_bfloat16, float>(p, tiles, pdl, stream)
                                   : launch<kWeightGrad, Ctas, BN, __half, float>(p, tiles, pdl, stream);
  return a.act_dtype == MFR_BF16 ? launch<kWeightGrad, Ctas, BN, __nv_bfloat16, __nv_bfloat16>(p, tiles, pdl, stream)
                                 : launch<kWeightGrad, Ctas, BN, __half, __half>(p, tiles, pdl, stream);
}

}  // namespace

cudaError_t launch_expert_weight_grad(const mfr_expert_matmul_backward_args& a, cudaStream_t stream) {
  const int64_t size = a.d_weight_dtype == MFR_FP32 ? 4 : 2;
  if (a.num_rows == 0)
    return a.accumulate ? cudaSuccess : cudaMemsetAsync(a.d_weight, 0, static_cast<size_t>(a.E) * a.n_out * a.n_in * size, stream);
  Params p = {};
  const CUtensorMapDataType type = map_type(a.act_dtype);
  cudaError_t e = encode_rows(&p.a, type, a.d_out, a.n_out, a.num_rows, a.d_out_stride * 2, 64, kDepth);
  if (e == cudaSuccess) e = encode_rows(&p.b, type, a.rows, a.n_in, a.num_rows, a.rows_stride * 2, 64, kDepth);
  if (e == cudaSuccess)
    e = encode_weights(&p.d, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type, a.d_weight, a.n_in, a.n_out, a.E, a.n_in * size,
                       static_cast<int64_t>(a.n_out) * a.n_in * size, static_cast<int>(128 / size), kTileM);
  if (e != cudaSuccess) return e;
  p.offsets = a.expert_offsets;
  p.counts = a.expert_counts;
  p.E = a.E;
  p.R = static_cast<int32_t>(a.num_rows);
  p.n_m = a.n_out;
  p.n_n = a.n_in;
  p.accumulate = a.accumulate;
  p.test_extra = (a.flags & MFR_FLAG_TEST_STREAM_TIMEOUT) != 0;
  // A pair's tiles cost more of a turnaround and fewer copies.  Measured, 32 experts of 4096 x 4096: 128 rows each 181 us by one CTA
  // a tile and 311 by pairs, 256 rows 248 and 354, 384 to 483 rows 436 and 437, 512 rows 408 and 391, 768 rows 563 and 492.  The rows
  // of the call are the buffer's: more than the experts' by their alignment and by routes elsewhere, which moves the border down by as
  // much.  (With at most 128 rows of weights the pair's second CTA would have none.)
  const bool pair = a.num_rows >= int64_t{512} * a.E && a.n_out > kTileM;
  return pair ? launch_weights<2>(a, p, stream) : launch_weights<1>(a, p, stream);
}

cudaError_t read_expert_timeouts(unsigned int* count) { return cudaMemcpyFromSymbol(count, g_expert_wait_timeouts, sizeof(unsigned int)); }

}  // namespace mfr
