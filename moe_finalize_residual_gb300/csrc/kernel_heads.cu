// Per-head RMSNorm of queries and keys and their position rotation in one pass, and its gradients.
//
// A group of G lanes (the power of two from D / 16 on) takes one head at a time; each of its first D / 16
// lanes holds 16 elements as two 16-byte vectors, chosen so that both elements of every rotated pair lie in
// the same lane:
//   half style         vectors p and p + rot/16 (elements i and i + rot/2), then the unrotated rest in twos
//   interleaved style  vectors 2p and 2p + 1 (neighbouring elements)
// so the rotation needs no exchange, and a head's sum of squares takes log2(G) shuffles.  The elements are
// kept as the pairs' first and second elements (`a` and `b`), two to a packed FP32 register pair, so that all
// the arithmetic runs on packed operations.  A warp computes the sines and cosines of its token's pairs once, in
// shared memory, and turns every head of the token by them.
//
// The angle position * inv_freq is reduced without error: inv_freq / (2 pi) is held as a 64-bit fraction of
// a turn (24-bit significand times 1 / (2 pi) to 64 bits), so the product with the position, modulo 2^64, is
// the fraction of the turn, with an error of position * 2^-64 turns.
//
// Bound by HBM: forward reads and writes each element once; backward reads two and writes one.
#include "layer_launch.h"

namespace mfr {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kHeadThreads = 256;
constexpr int kHeadWarps = kHeadThreads / 32;

// How a launch cuts one kind's work (queries or keys).  A warp's groups take `1 << gpt_log2` heads of a token at a
// time (a round) and the warp as many tokens as that leaves groups for; a token's rounds are cut into `splits`
// ranges.  A task is a block of tokens and a range; the kind's warps walk the tasks.
struct HeadCut {
  int gpt_log2;
  int rounds;
  int splits;
  int blocks;     // CTAs of the kind
  int64_t tasks;
};

// CTAs [0, q.blocks) take the queries, the rest the keys.
struct HeadParams {
  mfr_head_norm_args a;
  HeadCut q, k;
};

// inv_freq / (2 pi) as a fraction of a turn times 2^64, modulo 2^64.
__device__ __forceinline__ uint64_t turn_of(float inv_freq) {
  const uint32_t bits = __float_as_uint(inv_freq);
  const int e = (bits >> 23) & 0xff;
  if (e == 0) return 0;  // zero, and subnormals (below 2^-126 turns a position)
  // inv_freq = m 2^(e - 150);  1 / (2 pi) = c 2^-66, c rounded to 64 bits
  const uint64_t m = (bits & 0x7fffffu) | 0x800000u, c = 0xA2F9836E4E44152AULL;
  const uint64_t hi = __umul64hi(m, c), lo = m * c;
  const int s = 152 - e;  // turns 2^64 = (m c) 2^-s
  uint64_t r;
  if (s >= 128)
    r = 0;
  else if (s >= 64)
    r = hi >> (s - 64);
  else if (s > 0)
    r = (hi << (64 - s)) | (lo >> s);
  else
    r = s > -64 ? lo << -s : 0;
  return (bits >> 31) ? 0 - r : r;
}

// Where a lane's two vectors lie, and its 8 pairs.
struct LaneMap {
  int off_a, off_b;  // element offsets of the vectors
  int pair0;         // the first of its 8 pairs
  int pairs;         // how many of the 8 are rotated
};

__device__ __forceinline__ LaneMap lane_map(int p, int rot, int style) {
  LaneMap m;
  m.pair0 = 8 * p;
  if (style == MFR_ROTARY_INTERLEAVED || 16 * p >= rot) {
    m.off_a = 16 * p;
    m.off_b = 16 * p + 8;
  } else {
    m.off_a = 8 * p;
    m.off_b = 8 * p + rot / 2;
  }
  m.pairs = min(8, max(0, rot / 2 - 8 * p));
  return m;
}

// Fills the CTA's table of turns (shared memory, rot / 2 entries).
__device__ __forceinline__ void fill_turns(const mfr_head_norm_args& a, uint64_t* table) {
  for (int i = threadIdx.x; i < a.rot / 2; i += blockDim.x) table[i] = turn_of(a.inv_freq[i]);
  __syncthreads();
}

__device__ __forceinline__ int64_t position_of(const mfr_head_norm_args& a, int64_t t) {
  return (a.flags & MFR_FLAG_POSITIONS_64) ? static_cast<const int64_t*>(a.positions)[t]
                                           : static_cast<const int32_t*>(a.positions)[t];
}

// The cosines and sines of a warp's tokens: entry [(token, j, p)] holds pairs 8p + 2j and 8p + 2j + 1 of the token.
template <int G>
using TurnCache = float4[32 / G][4][G];

// Fills a warp's cache: 1 and 0 for unrotated pairs, times rotary_scale else.  `pos`: the position of the lane's
// group's token (gpt groups a token).
template <int G>
__device__ __forceinline__ void fill_cache(const mfr_head_norm_args& a, const uint64_t* table, int64_t pos, int gpt_log2, int lane,
                                           TurnCache<G>& cache) {
  const int entries = ((32 / G) >> gpt_log2) * 4 * G;
  __syncwarp();  // the last task's turns are done with
#pragma unroll 1
  for (int first = 0; first < entries; first += 32) {
    const int i = first + lane, token = i / (4 * G), j = i / G % 4, p = i % G;
    const int64_t at = __shfl_sync(kAll, pos, ((token << gpt_log2) * G) & 31);
    if (i >= entries) break;  // (the last iteration)
    float c[2], s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      c[k] = 1.0f;
      s[k] = 0.0f;
      const int pair = 8 * p + 2 * j + k;
      if (pair < a.rot / 2) {
        const uint64_t u = table[pair] * static_cast<uint64_t>(at);
        // the nearest 2^-32 turn, as a half turn in [-1, 1)
        const float h = static_cast<float>(static_cast<int32_t>((u + 0x80000000ULL) >> 32)) * 4.656612873077393e-10f;
        sincospif(h, &s[k], &c[k]);
        c[k] *= a.rotary_scale;
        s[k] *= a.rotary_scale;
      }
    }
    cache[token][j][p] = make_float4(c[0], c[1], s[0], s[1]);
  }
  __syncwarp();
}

// A lane's 16 elements of a head as they lie in memory, and as its pairs' first and second elements.
struct Raw {
  uint4 a, b;
};
struct Pairs {
  float2 a[4], b[4];
};

__device__ __forceinline__ Raw load_raw(const uint8_t* p, const LaneMap& m, bool on) {
  Raw r;
  r.a = on ? ldg16(p + 2 * m.off_a) : make_uint4(0, 0, 0, 0);
  r.b = on ? ldg16(p + 2 * m.off_b) : make_uint4(0, 0, 0, 0);
  return r;
}

template <typename A, int STYLE>
__device__ __forceinline__ Pairs unpack_pairs_of(const Raw& r) {
  Pairs v;
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (STYLE == MFR_ROTARY_HALF) {
      v.a[j] = Act<A>::unpack(w[j]);
      v.b[j] = Act<A>::unpack(w[j + 4]);
    } else {
      const float2 p = Act<A>::unpack(w[2 * j]), q = Act<A>::unpack(w[2 * j + 1]);
      v.a[j] = make_float2(p.x, q.x);
      v.b[j] = make_float2(p.y, q.y);
    }
  }
  return v;
}

template <typename A, int STYLE>
__device__ __forceinline__ void store_pairs(uint8_t* p, const LaneMap& m, const Pairs& v) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (STYLE == MFR_ROTARY_HALF) {
      w[j] = Act<A>::pack(v.a[j].x, v.a[j].y);
      w[j + 4] = Act<A>::pack(v.b[j].x, v.b[j].y);
    } else {
      w[2 * j] = Act<A>::pack(v.a[j].x, v.b[j].x);
      w[2 * j + 1] = Act<A>::pack(v.a[j].y, v.b[j].y);
    }
  }
  *reinterpret_cast<uint4*>(p + 2 * m.off_a) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + 2 * m.off_b) = make_uint4(w[4], w[5], w[6], w[7]);
}

// A kind's weight (ones without one) as each lane's pairs, in shared memory: [4][lanes of a head] vectors of (a, b)
// pairs, read without bank conflicts.  Threads first .. first + D / 16 - 1 of the CTA fill it.
using WeightTable = float4[4][MFR_MAX_HEAD_DIM / 16];
template <typename A, int STYLE>
__device__ __forceinline__ void fill_weight(const mfr_head_norm_args& a, const void* w, int first, WeightTable& table) {
  const int lane = static_cast<int>(threadIdx.x) - first;
  if (lane < 0 || lane >= a.D / 16) return;
  Pairs v;
  if (w != nullptr) {
    v = unpack_pairs_of<A, STYLE>(load_raw(static_cast<const uint8_t*>(w), lane_map(lane, a.rot, STYLE), true));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v.a[j] = v.b[j] = make_float2(1.0f, 1.0f);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) table[j][lane] = make_float4(v.a[j].x, v.a[j].y, v.b[j].x, v.b[j].y);
}

// Turns a lane's pairs by the angle, or back; `turn`: the token's cache at the lane, G entries apart.
template <bool BACK, int G>
__device__ __forceinline__ void turn_pairs(Pairs& v, const float4* turn) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 t = turn[j * G];
    const float2 c = make_float2(t.x, t.y), s = make_float2(t.z, t.w), a = v.a[j], b = v.b[j];
    const float2 ac = __fmul2_rn(a, c), bc = __fmul2_rn(b, c);
    if constexpr (BACK) {
      v.a[j] = __ffma2_rn(b, s, ac);
      v.b[j] = make_float2(__fmaf_rn(-a.x, s.x, bc.x), __fmaf_rn(-a.y, s.y, bc.y));
    } else {
      v.a[j] = make_float2(__fmaf_rn(-b.x, s.x, ac.x), __fmaf_rn(-b.y, s.y, ac.y));
      v.b[j] = __ffma2_rn(a, s, bc);
    }
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// 1 / sqrt(sum / D + eps): the norm's statistic in FP32, within 2 ulp of the root.
__device__ __forceinline__ float rstd_of(float sum, float inv_d, float eps) { return rsqrtf(__fmaf_rn(sum, inv_d, eps)); }

#ifndef HEADS_KB
#define HEADS_KB 4
#endif

// A warp's place in its kind's tasks: the token and the rounds of the current one.
struct Place {
  int64_t t;
  int64_t pos;  // -1 behind the last token
  int r0, r1;
};
template <int G>
__device__ __forceinline__ Place place_of(const mfr_head_norm_args& a, const HeadCut& cut, int64_t task, int group) {
  Place q;
  int split = 0;
  int64_t block = task;
  if (cut.splits > 1) {
    block = task / cut.splits;
    split = static_cast<int>(task - block * cut.splits);
  }
  q.t = block * ((32 / G) >> cut.gpt_log2) + (group >> cut.gpt_log2);
  q.r0 = cut.splits > 1 ? static_cast<int>(static_cast<int64_t>(cut.rounds) * split / cut.splits) : 0;
  q.r1 = cut.splits > 1 ? static_cast<int>(static_cast<int64_t>(cut.rounds) * (split + 1) / cut.splits) : cut.rounds;
  q.pos = task < cut.tasks && q.t < a.T ? position_of(a, q.t) : -1;
  return q;
}

// The lane's vectors of its group's head in round r of a place.
__device__ __forceinline__ int64_t head_at(const mfr_heads& h, const Place& q, int r, int gpt_log2, int sub) {
  return 2 * (q.t * h.token_stride + ((static_cast<int64_t>(r) << gpt_log2) + sub) * h.head_stride);
}

// Forward.  The next round's vectors (of the next task after a task's last round) are in flight while one is worked on.
template <typename A, int G, int STYLE>
__global__ void __launch_bounds__(kHeadThreads, HEADS_KB) head_norm_kernel(const __grid_constant__ HeadParams p) {
  __shared__ uint64_t table[MFR_MAX_HEAD_DIM / 2];
  __shared__ WeightTable weight;
  __shared__ TurnCache<G> caches[kHeadWarps];
  const mfr_head_norm_args& a = p.a;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = lane / G;
  const bool on = lane % G < a.D / 16;
  const LaneMap m = lane_map(lane % G, a.rot, STYLE);
  const bool keys = static_cast<int>(blockIdx.x) >= p.q.blocks;
  const HeadCut& cut = keys ? p.k : p.q;
  const int heads = keys ? a.k_heads : a.q_heads;
  const mfr_heads& in = keys ? a.k : a.q;
  const mfr_heads& out = keys ? a.k_out : a.q_out;
  const int gl = cut.gpt_log2, sub = group & ((1 << gl) - 1);
  const float4* turn = &caches[wid][group >> gl][0][lane % G];
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int64_t step = static_cast<int64_t>(cut.blocks) * kHeadWarps;
  int64_t task = static_cast<int64_t>(blockIdx.x - (keys ? p.q.blocks : 0)) * kHeadWarps + wid;
  pdl_launch_dependents();
  pdl_wait();
  Place q = place_of<G>(a, cut, task, group);
  const uint8_t* src = static_cast<const uint8_t*>(in.data);
  uint8_t* dst = static_cast<uint8_t*>(out.data);
  auto live = [&](const Place& z, int r) { return on && z.pos >= 0 && (r << gl) + sub < heads; };
  Raw raw = load_raw(src + head_at(in, q, q.r0, gl, sub), m, live(q, q.r0));
  fill_weight<A, STYLE>(a, keys ? a.k_weight : a.q_weight, 0, weight);
  fill_turns(a, table);
  const int64_t src_step = 2 * in.head_stride << gl, dst_step = 2 * out.head_stride << gl;
  while (task < cut.tasks) {
    task += step;
    const Place next = place_of<G>(a, cut, task, group);
    fill_cache<G>(a, table, q.pos, gl, lane, caches[wid]);
    const uint8_t* sp = src + head_at(in, q, q.r0, gl, sub);
    uint8_t* dp = dst + head_at(out, q, q.r0, gl, sub);
    for (int r = q.r0; r < q.r1; ++r) {  // the same trip count for the whole warp
      Pairs v = unpack_pairs_of<A, STYLE>(raw);
      sp += src_step;
      if (r + 1 == q.r1) {
        raw = load_raw(src + head_at(in, next, next.r0, gl, sub), m, live(next, next.r0));
      } else {
        raw = load_raw(sp, m, live(q, r + 1));
      }
      float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sq = __ffma2_rn(v.a[j], v.a[j], sq);
        sq = __ffma2_rn(v.b[j], v.b[j], sq);
      }
      const float rs = rstd_of(group_sum<G>(sq.x + sq.y), inv_d, a.eps);
      const float2 rr = make_float2(rs, rs);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w = weight[j][lane % G];
        v.a[j] = __fmul2_rn(__fmul2_rn(v.a[j], rr), make_float2(w.x, w.y));
        v.b[j] = __fmul2_rn(__fmul2_rn(v.b[j], rr), make_float2(w.z, w.w));
      }
      turn_pairs<false, G>(v, turn);
      if (live(q, r)) {
        store_pairs<A, STYLE>(dp, m, v);
      } else if ((a.flags & MFR_FLAG_ZERO_PADDING) && on && q.t < a.T && (r << gl) + sub < heads) {
        *reinterpret_cast<uint4*>(dp + 2 * m.off_a) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(dp + 2 * m.off_b) = make_uint4(0, 0, 0, 0);
      }
      dp += dst_step;
    }
    q = next;
  }
}

// Gradient: as forward, with the lanes' share of the weight gradient in registers; each CTA leaves one row of partial
// sums in the workspace.
template <typename A, int G, int STYLE>
__global__ void __launch_bounds__(kHeadThreads, 2) head_norm_grad_kernel(const __grid_constant__ HeadParams p) {
  extern __shared__ float part[];  // [kHeadWarps][D]
  __shared__ uint64_t table[MFR_MAX_HEAD_DIM / 2];
  __shared__ WeightTable weight;
  __shared__ TurnCache<G> caches[kHeadWarps];
  const mfr_head_norm_args& a = p.a;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = lane / G;
  const bool on = lane % G < a.D / 16;
  const LaneMap m = lane_map(lane % G, a.rot, STYLE);
  const bool keys = static_cast<int>(blockIdx.x) >= p.q.blocks;
  const HeadCut& cut = keys ? p.k : p.q;
  const int heads = keys ? a.k_heads : a.q_heads;
  const mfr_heads& in = keys ? a.k : a.q;
  const mfr_heads& out = keys ? a.k_out : a.q_out;
  const mfr_heads& dout = keys ? a.d_k_out : a.d_q_out;
  const int gl = cut.gpt_log2, sub = group & ((1 << gl) - 1);
  const float4* turn = &caches[wid][group >> gl][0][lane % G];
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int64_t step = static_cast<int64_t>(cut.blocks) * kHeadWarps;
  int64_t task = static_cast<int64_t>(blockIdx.x - (keys ? p.q.blocks : 0)) * kHeadWarps + wid;
  pdl_launch_dependents();
  pdl_wait();
  Place q = place_of<G>(a, cut, task, group);
  const uint8_t* x_src = static_cast<const uint8_t*>(in.data);
  const uint8_t* g_src = static_cast<const uint8_t*>(dout.data);
  uint8_t* dst = static_cast<uint8_t*>(out.data);
  auto live = [&](const Place& z, int r) { return on && z.pos >= 0 && (r << gl) + sub < heads; };
  Raw xr = load_raw(x_src + head_at(in, q, q.r0, gl, sub), m, live(q, q.r0));
  Raw gr = load_raw(g_src + head_at(dout, q, q.r0, gl, sub), m, live(q, q.r0));
  fill_weight<A, STYLE>(a, keys ? a.k_weight : a.q_weight, 0, weight);
  fill_turns(a, table);
  Pairs dw;
#pragma unroll
  for (int j = 0; j < 4; ++j) dw.a[j] = dw.b[j] = make_float2(0.0f, 0.0f);
  const int64_t x_step = 2 * in.head_stride << gl, g_step = 2 * dout.head_stride << gl, o_step = 2 * out.head_stride << gl;
  while (task < cut.tasks) {
    task += step;
    const Place next = place_of<G>(a, cut, task, group);
    fill_cache<G>(a, table, q.pos, gl, lane, caches[wid]);
    const uint8_t* xp = x_src + head_at(in, q, q.r0, gl, sub);
    const uint8_t* gp = g_src + head_at(dout, q, q.r0, gl, sub);
    uint8_t* op = dst + head_at(out, q, q.r0, gl, sub);
    for (int r = q.r0; r < q.r1; ++r) {
      const Pairs x = unpack_pairs_of<A, STYLE>(xr);
      Pairs g = unpack_pairs_of<A, STYLE>(gr);
      xp += x_step;
      gp += g_step;
      if (r + 1 == q.r1) {
        xr = load_raw(x_src + head_at(in, next, next.r0, gl, sub), m, live(next, next.r0));
        gr = load_raw(g_src + head_at(dout, next, next.r0, gl, sub), m, live(next, next.r0));
      } else {
        xr = load_raw(xp, m, live(q, r + 1));
        gr = load_raw(gp, m, live(q, r + 1));
      }
      turn_pairs<true, G>(g, turn);
      // sums of x^2 and of (g w) x
      float2 sq = make_float2(0.0f, 0.0f), dot = make_float2(0.0f, 0.0f);
      Pairs gw;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w = weight[j][lane % G];
        gw.a[j] = __fmul2_rn(g.a[j], make_float2(w.x, w.y));
        gw.b[j] = __fmul2_rn(g.b[j], make_float2(w.z, w.w));
        sq = __ffma2_rn(x.a[j], x.a[j], sq);
        sq = __ffma2_rn(x.b[j], x.b[j], sq);
        dot = __ffma2_rn(gw.a[j], x.a[j], dot);
        dot = __ffma2_rn(gw.b[j], x.b[j], dot);
      }
      const float rs = rstd_of(group_sum<G>(sq.x + sq.y), inv_d, a.eps);
      const float c = group_sum<G>(dot.x + dot.y) * inv_d * rs * rs * rs;
      const float2 rr = make_float2(rs, rs), cc = make_float2(-c, -c);
      Pairs d;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (a padding token's x and g are zeros)
        dw.a[j] = __ffma2_rn(g.a[j], __fmul2_rn(x.a[j], rr), dw.a[j]);
        dw.b[j] = __ffma2_rn(g.b[j], __fmul2_rn(x.b[j], rr), dw.b[j]);
        d.a[j] = __ffma2_rn(x.a[j], cc, __fmul2_rn(gw.a[j], rr));
        d.b[j] = __ffma2_rn(x.b[j], cc, __fmul2_rn(gw.b[j], rr));
      }
      if (on && q.t < a.T && (r << gl) + sub < heads) {
        if (q.pos < 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) d.a[j] = d.b[j] = make_float2(0.0f, 0.0f);
        }
        store_pairs<A, STYLE>(op, m, d);
      }
      op += o_step;
    }
    q = next;
  }
  if ((keys ? a.d_k_weight : a.d_q_weight) == nullptr) return;
  // over the warp's groups (lanes G apart), then over the CTA's warps in order
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int o = 16; o >= G; o >>= 1) {
      dw.a[j].x += __shfl_xor_sync(kAll, dw.a[j].x, o);
      dw.a[j].y += __shfl_xor_sync(kAll, dw.a[j].y, o);
      dw.b[j].x += __shfl_xor_sync(kAll, dw.b[j].x, o);
      dw.b[j].y += __shfl_xor_sync(kAll, dw.b[j].y, o);
    }
  }
  if (group == 0 && on) {
    float* row = part + wid * a.D;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (STYLE == MFR_ROTARY_HALF) {
        row[m.off_a + 2 * j] = dw.a[j].x;
        row[m.off_a + 2 * j + 1] = dw.a[j].y;
        row[m.off_b + 2 * j] = dw.b[j].x;
        row[m.off_b + 2 * j + 1] = dw.b[j].y;
      } else {
        row[m.off_a + 4 * j] = dw.a[j].x;
        row[m.off_a + 4 * j + 1] = dw.b[j].x;
        row[m.off_a + 4 * j + 2] = dw.a[j].y;
        row[m.off_a + 4 * j + 3] = dw.b[j].y;
      }
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += kHeadThreads) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeadWarps; ++i) s += part[i * a.D + d];
    static_cast<float*>(a.workspace)[static_cast<int64_t>(blockIdx.x) * a.D + d] = s;
  }
}

// Adds the partial weight gradients: CTA (kind, 32 elements), 32 rows at a time, then over the rows' warps
// in order.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) head_weight_grad_kernel(const __grid_constant__ HeadParams p) {
  __shared__ float part[32][33];
  const mfr_head_norm_args& a = p.a;
  pdl_launch_dependents();
  pdl_wait();
  const int parts = (a.D + 31) / 32;
  const bool keys = static_cast<int>(blockIdx.x) >= parts;
  float* out = keys ? a.d_k_weight : a.d_q_weight;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int d = (blockIdx.x % parts) * 32 + lane;
  const int64_t b0 = keys ? p.q.blocks : 0, b1 = p.q.blocks + (keys ? p.k.blocks : 0);
  float s = 0.0f;
  if (d < a.D) {
#pragma unroll 4
    for (int64_t b = b0 + wid; b < b1; b += 32) s += static_cast<const float*>(a.workspace)[b * a.D + d];
  }
  part[wid][lane] = s;
  __syncthreads();
  const float v = warp_sum(part[lane][wid]);
  if (lane == 0 && (blockIdx.x % parts) * 32 + wid < a.D) out[(blockIdx.x % parts) * 32 + wid] = v;
}

template <typename A, int G, int STYLE>
cudaError_t launch_forward(const HeadParams& p, int blocks, cudaStream_t stream) {
  return launch_pdl<HeadParams>(head_norm_kernel<A, G, STYLE>, dim3(blocks), kHeadThreads, 0, p.a.flags & MFR_FLAG_PDL, stream, p);
}
template <typename A, int G, int STYLE>
cudaError_t launch_backward(const HeadParams& p, int blocks, cudaStream_t stream) {
  return launch_pdl<HeadParams>(head_norm_grad_kernel<A, G, STYLE>, dim3(blocks), kHeadThreads, kHeadWarps * p.a.D * 4,
                                p.a.flags & MFR_FLAG_PDL, stream, p);
}

template <typename A, int STYLE>
cudaError_t launch_g(const HeadParams& p, int blocks, bool backward, cudaStream_t stream) {
  const int lanes = p.a.D / 16;
#define MFR_HEADS(G) \
  if (lanes <= G) return backward ? launch_backward<A, G, STYLE>(p, blocks, stream) : launch_forward<A, G, STYLE>(p, blocks, stream)
  MFR_HEADS(1);
  MFR_HEADS(2);
  MFR_HEADS(4);
  MFR_HEADS(8);
  MFR_HEADS(16);
  MFR_HEADS(32);
#undef MFR_HEADS
  return cudaErrorInvalidValue;
}

template <typename A>
cudaError_t launch_s(const HeadParams& p, int blocks, bool backward, cudaStream_t stream) {
  return p.a.style == MFR_ROTARY_HALF ? launch_g<A, MFR_ROTARY_HALF>(p, blocks, backward, stream)
                                      : launch_g<A, MFR_ROTARY_INTERLEAVED>(p, blocks, backward, stream);
}

int groups_of(int D) {
  int g = 1;
  while (g < D / 16) g *= 2;
  return 32 / g;
}

int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Cuts one kind's heads for at most `most` CTAs: as many groups on a token as it has heads for, and a token's rounds
// in more ranges when the tokens alone leave warps idle.
HeadCut cut_heads(int T, int heads, int groups, int64_t most) {
  HeadCut c{};
  if (heads == 0 || T == 0) return c;
  while ((2 << c.gpt_log2) <= groups && (2 << c.gpt_log2) <= heads) ++c.gpt_log2;
  c.rounds = static_cast<int>(ceil_div64(heads, 1 << c.gpt_log2));
  const int64_t blocks = ceil_div64(T, groups >> c.gpt_log2);
  int64_t splits = most * kHeadWarps / blocks;
  if (splits > c.rounds) splits = c.rounds;
  if (splits < 1) splits = 1;
  c.splits = static_cast<int>(splits);
  c.tasks = blocks * splits;
  const int64_t want = ceil_div64(c.tasks, kHeadWarps);
  c.blocks = static_cast<int>(want < most ? want : most);
  return c;
}

// Shares `blocks` CTAs between the kinds in proportion to their work: a token's rounds, and its turns (about one
// round's work); at least one for each kind that has heads.
HeadParams cut_kinds(const mfr_head_norm_args& a, int blocks) {
  HeadParams p{a, {}, {}};
  const int groups = groups_of(a.D);
  const int64_t wq = a.q_heads > 0 ? ceil_div64(a.q_heads, groups) + 1 : 0, wk = a.k_heads > 0 ? ceil_div64(a.k_heads, groups) + 1 : 0;
  int64_t q = blocks * wq / (wq + wk);
  if (a.q_heads > 0 && q == 0) q = 1;
  if (a.k_heads > 0 && q == blocks) q = blocks - 1;
  p.q = cut_heads(a.T, a.q_heads, groups, q);
  p.k = cut_heads(a.T, a.k_heads, groups, blocks - q);
  return p;
}

}  // namespace

cudaError_t launch_head_norm(const mfr_head_norm_args& a, cudaStream_t stream) {
  const HeadParams p = cut_kinds(a, 152 * HEADS_KB);
  const int blocks = p.q.blocks + p.k.blocks;
  return a.act_dtype == MFR_BF16 ? launch_s<__nv_bfloat16>(p, blocks, false, stream) : launch_s<__half>(p, blocks, false, stream);
}

cudaError_t launch_head_norm_backward(const mfr_head_norm_args& a, cudaStream_t stream) {
  const HeadParams p = cut_kinds(a, kHeadGradBlocks);
  cudaError_t e = cudaSuccess;
  const int blocks = p.q.blocks + p.k.blocks;
  if (a.T > 0) e = a.act_dtype == MFR_BF16 ? launch_s<__nv_bfloat16>(p, blocks, true, stream) : launch_s<__half>(p, blocks, true, stream);
  // (no tokens: no partial sums, and the weight gradients are zeros)
  if (e != cudaSuccess || (a.d_q_weight == nullptr && a.d_k_weight == nullptr)) return e;
  return launch_pdl<HeadParams>(head_weight_grad_kernel, dim3(2 * ((a.D + 31) / 32)), kSumThreads, 0, a.flags & MFR_FLAG_PDL, stream, p);
}

}  // namespace mfr
