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
// The angle position * inv_freq is reduced in integers: inv_freq / (2 pi) is held as a 128-bit fraction of a turn
// (24-bit significand times 1 / (2 pi) to 128 bits), and the first 64 bits of its product with the position, modulo
// 2^128, are the fraction of the turn: within 2^-47 of a turn for any 64-bit position and |inv_freq| < 2^20.  32-bit
// positions make do with the first 64 bits of inv_freq's turn, within 2^-33.  The sine and cosine take the nearest 2^-32.
//
// The work is cut into rounds: one head for each of a warp's groups.  A warp keeps the vectors of its next rounds in
// flight by cp.async into slots of shared memory that each lane fills and reads by itself, so no warp waits for
// another.
//
// Bound by HBM: forward reads and writes each element once; backward reads two and writes one.  Measured on GB300 (copy
// bandwidth 6779 GB/s), 48 + 8 heads of 128, BF16, from a packed projection: forward of 16384 tokens, 470 MB, 71.7 us
// (0.97 of the copy); gradient of 8192 tokens, 352 MB, 60.5 us (0.86), of which 3 us are the sum of the weight gradients.
#include <algorithm>

#include "layer_launch.h"

namespace mfr {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// How a launch cuts its work.  A warp's groups take `1 << gpt_log2` heads of a token at a time (a round: first the
// queries', then the keys') and the warp as many tokens (a block) as that leaves groups for.  Forward, `splits` warps
// share a block's rounds; backward, all `warps` share all blocks' rounds.
struct HeadCut {
  int gpt_log2;
  int q_rounds, k_rounds;
  int splits;
  int cache_bytes;      // a warp's turn cache
  int64_t blocks;       // of tokens
  int64_t warps;
  int64_t ctas;
};

struct HeadParams {
  mfr_head_norm_args a;
  HeadCut cut;
};

// position * inv_freq / (2 pi) as a fraction of a turn times 2^64, modulo 2^64, for |inv_freq| < 2^20.
__device__ __forceinline__ uint64_t turns_of(float inv_freq, int64_t pos, bool wide) {
  const uint32_t bits = __float_as_uint(inv_freq);
  const int e = (bits >> 23) & 0xff;
  if (e == 0) return 0;  // zero, and subnormals (below 2^-126 turns a position)
  // inv_freq = m 2^(e - 150);  1 / (2 pi) = (c1 2^64 + c0) 2^-130, to 128 bits;  m (c1 2^64 + c0) = t1 2^128 + t0 2^64 + low
  const uint64_t m = (bits & 0x7fffffu) | 0x800000u, c1 = 0xA2F9836E4E441529ULL, c0 = 0xFC2757D1F534DDC1ULL;
  const uint64_t low = m * c0, carry = __umul64hi(m, c0), t0 = m * c1 + carry, t1 = __umul64hi(m, c1) + (t0 < carry ? 1 : 0);
  // a position's turns times 2^128 are that times 2^-s: hi 2^64 + lo, modulo 2^128
  const int s = max(152 - e, 1), k = s & 63;  // (s >= 6 for the frequencies allowed)
  const uint64_t n = static_cast<uint64_t>(pos), hi = s < 64 ? (t1 << (64 - s)) | (t0 >> s) : s < 128 ? t1 >> k : 0;
  uint64_t u = hi * n;
  if (wide) {  // (times a position below 2^31, lo is less than 2^-33 of a turn)
    const uint64_t up = k == 0 ? 0 : s < 64 ? t0 << (64 - k) : t1 << (64 - k);
    u += __umul64hi(s < 64 ? up | (low >> s) : s < 128 ? up | (t0 >> k) : t1 >> k, n);
  }
  return (bits >> 31) ? 0 - u : u;
}

// Where a lane's two vectors lie, and how many of its 8 pairs are rotated.
struct LaneMap {
  int off_a, off_b;  // element offsets of the vectors
  int pairs;
};

__device__ __forceinline__ LaneMap lane_map(int p, int rot, int style) {
  LaneMap m;
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

// Of the pairs 2j and 2j + 1 the turned element where the pair is rotated, else the one that passes: a turn by (1, 0) would
// add zero times its partner, which may be an infinity or NaN.
__device__ __forceinline__ float2 rotated_of(const LaneMap& m, int j, float2 turned, float2 passed) {
  return make_float2(2 * j < m.pairs ? turned.x : passed.x, 2 * j + 1 < m.pairs ? turned.y : passed.y);
}

__device__ __forceinline__ int64_t position_of(const mfr_head_norm_args& a, int64_t t) {
  return (a.flags & MFR_FLAG_POSITIONS_64) ? static_cast<const int64_t*>(a.positions)[t]
                                           : static_cast<const int32_t*>(a.positions)[t];
}

// The cosine and sine of the angle at a position, times `scale`; `wide`: the position may be 2^31 or more.
__device__ __forceinline__ float2 cos_sin(float inv_freq, int64_t pos, bool wide, float scale) {
  const uint64_t u = turns_of(inv_freq, pos, wide);
  // the nearest 2^-32 turn, as a half turn in [-1, 1)
  const float h = static_cast<float>(static_cast<int32_t>((u + 0x80000000ULL) >> 32)) * 4.656612873077393e-10f;
  float s, c;
  sincospif(h, &s, &c);
  return make_float2(c * scale, s * scale);
}

// A lane's 16 elements of a head as they lie in memory, and as its pairs' first and second elements.
struct Raw {
  uint4 a, b;
};
struct Pairs {
  float2 a[4], b[4];
};

__device__ __forceinline__ Raw load_raw(const uint8_t* p, const LaneMap& m) { return {ldg16(p + 2 * m.off_a), ldg16(p + 2 * m.off_b)}; }

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
__device__ __forceinline__ void store_pairs(uint8_t* p, int second, const Pairs& v) {
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
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + second) = make_uint4(w[4], w[5], w[6], w[7]);
}


// What a warp's tokens turn by, in shared memory: for lane p of a head and its pairs 2j and 2j + 1 two vectors that fold
// the weight in, so that the rotation of the normed head is  a' = a A1 + b A2,  b' = b B1 + a B2:
//   [kind][token][j][0][p] = A1 = c w_a, A2 = -s w_b      [..][1][p] = B1 = c w_b, B2 = s w_a      (two pairs each)
template <int G>
using TurnCache = float4 (*)[4][2][G];

// A weight's elements of a pair (ones without a weight).
template <typename A, int STYLE>
__device__ __forceinline__ float2 weight_pair(const void* w, int p, int k, const LaneMap& m) {
  if (w == nullptr) return make_float2(1.0f, 1.0f);
  // pair k of lane p: elements off_a + k and off_b + k, or off_a + 2k and off_a + 2k + 1
  const int e0 = STYLE == MFR_ROTARY_HALF ? m.off_a + k : m.off_a + 2 * k, e1 = STYLE == MFR_ROTARY_HALF ? m.off_b + k : e0 + 1;
  const A* v = static_cast<const A*>(w);
  return make_float2(static_cast<float>(v[e0]), static_cast<float>(v[e1]));
}

// Fills a warp's cache for its block of tokens; `pos`: the position of the lane's group's token.
template <typename A, int G, int STYLE>
__device__ __forceinline__ void fill_cache(const mfr_head_norm_args& a, int64_t pos, int gpt_log2, int lane, TurnCache<G> cache) {
  const int tokens = (32 / G) >> gpt_log2, entries = tokens * 4 * G;
#pragma unroll 1
  for (int first = 0; first < entries; first += 32) {
    const int i = first + lane, token = i / (4 * G), j = i / G % 4, p = i % G;
    const int64_t at = __shfl_sync(kAll, pos, ((token << gpt_log2) * G) & 31);
    if (i >= entries || p >= a.D / 16) continue;  // (the same trip count for all lanes)
    const LaneMap m = lane_map(p, a.rot, STYLE);
    float2 t[2];
    bool on[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int pair = 8 * p + 2 * j + k;
      on[k] = pair < a.rot / 2;
      t[k] = on[k] ? cos_sin(a.inv_freq[pair], at, a.flags & MFR_FLAG_POSITIONS_64, a.rotary_scale) : make_float2(1.0f, 0.0f);
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const void* weight = kind ? a.k_weight : a.q_weight;
      const float2 w0 = weight_pair<A, STYLE>(weight, p, 2 * j, m), w1 = weight_pair<A, STYLE>(weight, p, 2 * j + 1, m);
      auto entry = cache[kind * tokens + token][j];
      // (an element that passes has nothing of its partner's weight, whatever that is)
      entry[0][p] = make_float4(t[0].x * w0.x, t[1].x * w1.x, on[0] ? -t[0].y * w0.y : 0.0f, on[1] ? -t[1].y * w1.y : 0.0f);
      entry[1][p] = make_float4(t[0].x * w0.y, t[1].x * w1.y, on[0] ? t[0].y * w0.x : 0.0f, on[1] ? t[1].y * w1.x : 0.0f);
    }
  }
  __syncwarp();
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// 1 / sqrt(sum / D + eps): the norm's statistic in FP32, within 2 ulp of the root.
__device__ __forceinline__ float rstd_of(float sum, float inv_d, float eps) { return rsqrtf(__fmaf_rn(sum, inv_d, eps)); }

// A lane's way through the rounds of a block's queries and then keys: its first vector of its group's head.
struct Walk {
  uint8_t* at;
  uint8_t* keys;  // where the keys begin
  int64_t step, key_step;
  __device__ __forceinline__ void start(const mfr_heads& q, const mfr_heads& k, const HeadCut& cut, int64_t t, int sub, int offset, int r) {
    step = 2 * q.head_stride << cut.gpt_log2;
    key_step = 2 * k.head_stride << cut.gpt_log2;
    keys = static_cast<uint8_t*>(k.data) + 2 * (t * k.token_stride + sub * k.head_stride + offset);
    at = static_cast<uint8_t*>(q.data) + 2 * (t * q.token_stride + sub * q.head_stride + offset) + r * step;
    if (r >= cut.q_rounds) {
      at = keys + (r - cut.q_rounds) * key_step;
      step = key_step;
    }
  }
  // to round r + 1
  __device__ __forceinline__ void next(const HeadCut& cut, int r) {
    at += step;
    if (r + 1 == cut.q_rounds) {
      at = keys;
      step = key_step;
    }
  }
};

// Slots of a warp's rounds in flight: N vectors a lane and round, each lane its own.
template <int S, int N>
constexpr int kSlotBytes = S * N * 32 * 16;

constexpr int kFwdSlots = 4;
constexpr int kFwdThreads = 64;
constexpr int kFwdCtas = 12;  // CTAs an SM holds, by registers

// Forward: a warp takes its rounds of one block of tokens.  The CTAs are small and come and go, which evens out the
// SMs' load; a warp requests its first vectors, its position, frequencies and weights all at once.  Persistent warps
// with equal shares took 82 to 88 us for the 71.7 above: their streams lie far apart, or the last of them end late.
template <typename A, int G, int STYLE>
__global__ void __launch_bounds__(kFwdThreads, kFwdCtas) head_norm_kernel(const __grid_constant__ HeadParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const mfr_head_norm_args& a = p.a;
  const HeadCut& cut = p.cut;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = lane / G;
  const bool lane_on = lane % G < a.D / 16;  // the other lanes double the first one's vectors and count nothing
  const LaneMap m = lane_map(lane_on ? lane % G : 0, a.rot, STYLE);
  const int second = 2 * (m.off_b - m.off_a);
  const int gl = cut.gpt_log2, tokens = (32 / G) >> gl, sub = group & ((1 << gl) - 1);
  uint8_t* mine = smem + wid * (kSlotBytes<kFwdSlots, 2> + cut.cache_bytes);
  auto cache = reinterpret_cast<TurnCache<G>>(mine + kSlotBytes<kFwdSlots, 2>);
  const uint32_t slot = smem_addr(mine) + lane * 16;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kFwdThreads / 32) + wid;
  pdl_launch_dependents();
  pdl_wait();
  if (warp >= cut.warps) return;
  int64_t block = warp;
  int r0 = 0, r1 = cut.q_rounds + cut.k_rounds;
  if (cut.splits > 1) {
    block = warp / cut.splits;
    const int split = static_cast<int>(warp - block * cut.splits), all = r1;
    r0 = all * split / cut.splits;
    r1 = all * (split + 1) / cut.splits;
  }
  const int64_t t = block * tokens + (group >> gl);
  const bool in = t < a.T;
  // the rounds that the lane's group has heads for, of each kind
  const int q_last = (a.q_heads - sub + (1 << gl) - 1) >> gl, k_last = cut.q_rounds + ((a.k_heads - sub + (1 << gl) - 1) >> gl);
  Walk src, dst;
  src.start(a.q, a.k, cut, t, sub, m.off_a, r0);
  auto request = [&](int r, int to_slot) {
    if (r < r1) {
      const bool take = in && r < (r < cut.q_rounds ? q_last : k_last);
      const uint32_t to = slot + to_slot * (2 * 32 * 16);
      cp_async16_if(to, src.at, take);
      cp_async16_if(to + 32 * 16, src.at + second, take);
      src.next(cut, r);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kFwdSlots - 1; ++i) request(r0 + i, i);
  const int64_t pos = in ? position_of(a, t) : -1;
  dst.start(a.q_out, a.k_out, cut, t, sub, m.off_a, r0);
  fill_cache<A, G, STYLE>(a, pos, gl, lane, cache);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const bool write = lane_on && in && (pos >= 0 || (a.flags & MFR_FLAG_ZERO_PADDING));
  int here = 0;  // the slot of the current round
  for (int r = r0; r < r1; ++r) {  // the same trip count for the whole warp
    const float4* turn = &cache[(r < cut.q_rounds ? 0 : tokens) + (group >> gl)][0][0][lane % G];
    cp_async_wait_group<kFwdSlots - 2>();
    const uint32_t from = slot + here * (2 * 32 * 16);
    const Raw raw{lds16(from), lds16(from + 32 * 16)};
    request(r + kFwdSlots - 1, here == 0 ? kFwdSlots - 1 : here - 1);
    here = here + 1 == kFwdSlots ? 0 : here + 1;
    const Pairs x = unpack_pairs_of<A, STYLE>(raw);
    float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sq = __ffma2_rn(x.a[j], x.a[j], sq);
      sq = __ffma2_rn(x.b[j], x.b[j], sq);
    }
    const float rs = rstd_of(group_sum<G>(lane_on ? sq.x + sq.y : 0.0f), inv_d, a.eps);
    const float2 rr = make_float2(rs, rs);
    Pairs v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 ta = turn[2 * j * G], tb = turn[(2 * j + 1) * G];
      const float2 xa = __fmul2_rn(x.a[j], rr), xb = __fmul2_rn(x.b[j], rr);
      v.a[j] = __ffma2_rn(xb, make_float2(ta.z, ta.w), __fmul2_rn(xa, make_float2(ta.x, ta.y)));
      v.b[j] = __ffma2_rn(xa, make_float2(tb.z, tb.w), __fmul2_rn(xb, make_float2(tb.x, tb.y)));
    }
    if (rs == 0.0f) {
      // An element is infinite, or as good as that: zero times it must not reach a partner that passes.  (The elements are
      // taken from the slot again, so that the other heads keep no register for this.)
      const LaneMap again = lane_map(lane_on ? lane % G : 0, a.rot, STYLE);
      const Pairs y = unpack_pairs_of<A, STYLE>({lds16(from), lds16(from + 32 * 16)});
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 ta = turn[2 * j * G], tb = turn[(2 * j + 1) * G];
        v.a[j] = rotated_of(again, j, v.a[j], __fmul2_rn(__fmul2_rn(y.a[j], rr), make_float2(ta.x, ta.y)));
        v.b[j] = rotated_of(again, j, v.b[j], __fmul2_rn(__fmul2_rn(y.b[j], rr), make_float2(tb.x, tb.y)));
      }
    }
    if (write && r < (r < cut.q_rounds ? q_last : k_last)) {
      if (pos >= 0) {
        store_pairs<A, STYLE>(dst.at, second, v);
      } else {
        *reinterpret_cast<uint4*>(dst.at) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(dst.at + second) = make_uint4(0, 0, 0, 0);
      }
    }
    dst.next(cut, r);
  }
}


constexpr int kBwdSlots = 3;
constexpr int kBwdThreads = 192;
constexpr int kBwdCtas = 2;  // CTAs an SM holds: 12 warps of 168 registers (16 of 128 spill: 63.3 against 60.1 us)
constexpr int kBwdWarps = kBwdThreads / 32;

// A kind's weight as each lane's pairs, in shared memory: [4][lanes of a head] vectors of (a, b) pairs.
using WeightTable = float4[4][MFR_MAX_HEAD_DIM / 16];
template <typename A, int STYLE>
__device__ __forceinline__ void fill_weight(const mfr_head_norm_args& a, const void* w, int first, WeightTable& table) {
  const int lane = static_cast<int>(threadIdx.x) - first;
  if (lane < 0 || lane >= a.D / 16) return;
  Pairs v;
  if (w != nullptr) {
    v = unpack_pairs_of<A, STYLE>(load_raw(static_cast<const uint8_t*>(w), lane_map(lane, a.rot, STYLE)));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v.a[j] = v.b[j] = make_float2(1.0f, 1.0f);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) table[j][lane] = make_float4(v.a[j].x, v.a[j].y, v.b[j].x, v.b[j].y);
}

// What a warp's tokens turn by: [token][j][p], the cosines and the sines of pairs 2j and 2j + 1 of lane p.
template <int G>
__device__ __forceinline__ void fill_turns(const mfr_head_norm_args& a, int64_t pos, int gpt_log2, int lane, float4 (*cache)[4][G]) {
  const int entries = ((32 / G) >> gpt_log2) * 4 * G;
  __syncwarp();  // the last block's turns are done with
#pragma unroll 1
  for (int first = 0; first < entries; first += 32) {
    const int i = first + lane, token = i / (4 * G), j = i / G % 4, p = i % G;
    const int64_t at = __shfl_sync(kAll, pos, ((token << gpt_log2) * G) & 31);
    if (i >= entries) continue;
    float2 t[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int pair = 8 * p + 2 * j + k;
      t[k] = pair < a.rot / 2 ? cos_sin(a.inv_freq[pair], at, a.flags & MFR_FLAG_POSITIONS_64, a.rotary_scale) : make_float2(1.0f, 0.0f);
    }
    cache[token][j][p] = make_float4(t[0].x, t[1].x, t[0].y, t[1].y);
  }
  __syncwarp();
}

// Turns a lane's pairs back; `turn`: the token's turns at the lane.
template <int G>
__device__ __forceinline__ void turn_back(Pairs& v, const float4* turn) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 t = turn[j * G];
    const float2 c = make_float2(t.x, t.y), s = make_float2(t.z, t.w), a = v.a[j], b = v.b[j];
    const float2 bc = __fmul2_rn(b, c);
    v.a[j] = __ffma2_rn(b, s, __fmul2_rn(a, c));
    v.b[j] = make_float2(__fmaf_rn(-a.x, s.x, bc.x), __fmaf_rn(-a.y, s.y, bc.y));
  }
}

// Adds a lane's share of a weight gradient over the warp's groups (lanes G apart) and writes it to the warp's row.
template <int G, int STYLE>
__device__ __forceinline__ void write_sums(Pairs dw, const LaneMap& m, bool write, float* row) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int o = 16; o >= G; o >>= 1) {
      dw.a[j].x += __shfl_xor_sync(kAll, dw.a[j].x, o);
      dw.a[j].y += __shfl_xor_sync(kAll, dw.a[j].y, o);
      dw.b[j].x += __shfl_xor_sync(kAll, dw.b[j].x, o);
      dw.b[j].y += __shfl_xor_sync(kAll, dw.b[j].y, o);
    }
    if (write) {
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
}

// A warp's shared memory in the gradient: its slots (later its sums), its turns, and each lane's share of the keys'
// weight gradient (the queries' is in registers: they are the larger part).
constexpr int kKeySumBytes = 4 * 32 * 16;
__host__ __device__ constexpr int bwd_warp_bytes(int cache_bytes) { return kSlotBytes<kBwdSlots, 4> + cache_bytes + kKeySumBytes; }

// Gradient: the warps that the GPU holds share all rounds equally, each a contiguous range, so that few rows of partial
// weight gradients are left to add (CTAs that come and go, as forward: 57 us, but 6.5 us more to add their rows).
template <typename A, int G, int STYLE>
__global__ void __launch_bounds__(kBwdThreads, kBwdCtas) head_norm_grad_kernel(const __grid_constant__ HeadParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ WeightTable weights[2];
  const mfr_head_norm_args& a = p.a;
  const HeadCut& cut = p.cut;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = lane / G;
  const bool lane_on = lane % G < a.D / 16;
  const LaneMap m = lane_map(lane_on ? lane % G : 0, a.rot, STYLE);
  const int second = 2 * (m.off_b - m.off_a);
  const int gl = cut.gpt_log2, tokens = (32 / G) >> gl, sub = group & ((1 << gl) - 1);
  uint8_t* mine = smem + wid * bwd_warp_bytes(cut.cache_bytes);
  auto cache = reinterpret_cast<float4(*)[4][G]>(mine + kSlotBytes<kBwdSlots, 4>);
  float4* key_sums = reinterpret_cast<float4*>(mine + kSlotBytes<kBwdSlots, 4> + cut.cache_bytes) + lane;  // [4][32]
  const float4* turn = &cache[group >> gl][0][lane % G];
  const uint32_t slot = smem_addr(mine) + lane * 16;
  // the warp's rounds, an equal share of all blocks' rounds: from round r of a block on, `left` of them
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kBwdWarps + wid;
  const int all = cut.q_rounds + cut.k_rounds;
  const int64_t total = cut.blocks * all;
  int64_t left = 0, block = 0;
  int r = 0;
  if (warp < cut.warps) {
    const int64_t first = total / cut.warps * warp + min(total % cut.warps, warp);
    left = total / cut.warps + (warp < total % cut.warps ? 1 : 0);
    block = first / all;
    r = static_cast<int>(first - block * all);
  }
  const int q_last = (a.q_heads - sub + (1 << gl) - 1) >> gl, k_last = cut.q_rounds + ((a.k_heads - sub + (1 << gl) - 1) >> gl);
  pdl_launch_dependents();
  pdl_wait();
  auto token = [&](int64_t b) { return b * tokens + (group >> gl); };
  auto position = [&](int64_t b) { return token(b) < a.T ? position_of(a, token(b)) : -1; };
  Walk xs, gs, dst;
  int64_t next_block = block, next_left = left;
  int next_r = r;
  bool next_in = false, next_new = true;
  auto request = [&](int to_slot) {  // the next round, if there is one
    if (next_left > 0) {
      if (next_new) {
        next_in = token(next_block) < a.T;
        xs.start(a.q, a.k, cut, token(next_block), sub, m.off_a, next_r);
        gs.start(a.d_q_out, a.d_k_out, cut, token(next_block), sub, m.off_a, next_r);
        next_new = false;
      }
      const bool take = next_in && next_r < (next_r < cut.q_rounds ? q_last : k_last);
      const uint32_t to = slot + to_slot * (4 * 32 * 16);
      cp_async16_if(to, xs.at, take);
      cp_async16_if(to + 32 * 16, xs.at + second, take);
      cp_async16_if(to + 2 * 32 * 16, gs.at, take);
      cp_async16_if(to + 3 * 32 * 16, gs.at + second, take);
      xs.next(cut, next_r);
      gs.next(cut, next_r);
      --next_left;
      if (++next_r == all) {
        next_r = 0;
        ++next_block;
        next_new = true;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kBwdSlots - 1; ++i) request(i);
  int64_t pos_next = position(block);
  fill_weight<A, STYLE>(a, a.q_weight, 0, weights[0]);
  fill_weight<A, STYLE>(a, a.k_weight, 32, weights[1]);
  Pairs dw;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    dw.a[j] = dw.b[j] = make_float2(0.0f, 0.0f);
    key_sums[32 * j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  __syncthreads();
  const float inv_d = 1.0f / static_cast<float>(a.D);
  int here = 0;  // the slot of the current round
  for (; left > 0; ++block, r = 0) {
    const int64_t pos = pos_next;
    pos_next = position(block + 1);
    const bool write = lane_on && token(block) < a.T;
    dst.start(a.q_out, a.k_out, cut, token(block), sub, m.off_a, r);
    fill_turns<G>(a, pos, gl, lane, cache);
    for (; r < all && left > 0; ++r, --left) {
      const bool key = r >= cut.q_rounds;
      cp_async_wait_group<kBwdSlots - 2>();
      const uint32_t from = slot + here * (4 * 32 * 16);
      const Raw xr{lds16(from), lds16(from + 32 * 16)}, gr{lds16(from + 2 * 32 * 16), lds16(from + 3 * 32 * 16)};
      request(here == 0 ? kBwdSlots - 1 : here - 1);
      here = here + 1 == kBwdSlots ? 0 : here + 1;
      const Pairs x = unpack_pairs_of<A, STYLE>(xr);
      Pairs g = unpack_pairs_of<A, STYLE>(gr);
      turn_back<G>(g, turn);
      if (a.rot < a.D) {  // (from the slot again: no register is kept for this)
        const LaneMap again = lane_map(lane_on ? lane % G : 0, a.rot, STYLE);
        const Pairs y = unpack_pairs_of<A, STYLE>({lds16(from + 2 * 32 * 16), lds16(from + 3 * 32 * 16)});
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g.a[j] = rotated_of(again, j, g.a[j], y.a[j]);
          g.b[j] = rotated_of(again, j, g.b[j], y.b[j]);
        }
      }
      // sums of x^2 and of (g w) x
      float2 sq = make_float2(0.0f, 0.0f), dot = make_float2(0.0f, 0.0f);
      Pairs gw;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w = weights[key][j][lane % G];
        gw.a[j] = __fmul2_rn(g.a[j], make_float2(w.x, w.y));
        gw.b[j] = __fmul2_rn(g.b[j], make_float2(w.z, w.w));
        sq = __ffma2_rn(x.a[j], x.a[j], sq);
        sq = __ffma2_rn(x.b[j], x.b[j], sq);
        dot = __ffma2_rn(gw.a[j], x.a[j], dot);
        dot = __ffma2_rn(gw.b[j], x.b[j], dot);
      }
      const float rs = rstd_of(group_sum<G>(lane_on ? sq.x + sq.y : 0.0f), inv_d, a.eps);
      const float c = group_sum<G>(lane_on ? dot.x + dot.y : 0.0f) * inv_d * rs * rs * rs;
      const float2 rr = make_float2(rs, rs), cc = make_float2(-c, -c);
      if (write && r < (key ? k_last : q_last)) {
        Pairs d;
        if (pos >= 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 xa = __fmul2_rn(x.a[j], rr), xb = __fmul2_rn(x.b[j], rr);
            if (!key) {
              dw.a[j] = __ffma2_rn(g.a[j], xa, dw.a[j]);
              dw.b[j] = __ffma2_rn(g.b[j], xb, dw.b[j]);
            } else {
              const float4 s = key_sums[32 * j];
              const float2 sa = __ffma2_rn(g.a[j], xa, make_float2(s.x, s.y)), sb = __ffma2_rn(g.b[j], xb, make_float2(s.z, s.w));
              key_sums[32 * j] = make_float4(sa.x, sa.y, sb.x, sb.y);
            }
            d.a[j] = __ffma2_rn(x.a[j], cc, __fmul2_rn(gw.a[j], rr));
            d.b[j] = __ffma2_rn(x.b[j], cc, __fmul2_rn(gw.b[j], rr));
          }
        } else {  // a padding token, whatever it holds
#pragma unroll
          for (int j = 0; j < 4; ++j) d.a[j] = d.b[j] = make_float2(0.0f, 0.0f);
        }
        store_pairs<A, STYLE>(dst.at, second, d);
      }
      dst.next(cut, r);
    }
  }
  if (a.d_q_weight == nullptr && a.d_k_weight == nullptr) return;
  // over the warp's groups, then over the CTA's warps in order
  cp_async_wait_all();
  __syncwarp();
  float* row = reinterpret_cast<float*>(mine);  // [2][D], in place of the slots
  write_sums<G, STYLE>(dw, m, lane_on && group == 0, row);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 s = key_sums[32 * j];
    dw.a[j] = make_float2(s.x, s.y);
    dw.b[j] = make_float2(s.z, s.w);
  }
  write_sums<G, STYLE>(dw, m, lane_on && group == 0, row + a.D);
  __syncthreads();
  for (int d = threadIdx.x; d < 2 * a.D; d += kBwdThreads) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kBwdWarps; ++i) s += reinterpret_cast<const float*>(smem + i * bwd_warp_bytes(cut.cache_bytes))[d];
    static_cast<float*>(a.workspace)[static_cast<int64_t>(blockIdx.x) * 2 * a.D + d] = s;
  }
}

// Adds the CTAs' partial weight gradients: a CTA takes 8 columns of the [2][D] rows, a warp 4 rows at a time; the sums
// meet by a butterfly over the lanes of a column and then over the warps in order.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) head_weight_grad_kernel(const __grid_constant__ HeadParams p) {
  __shared__ float part[kSumThreads / 32][8];
  const mfr_head_norm_args& a = p.a;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int d = blockIdx.x * 8 + (lane & 7);
  float* out = d < a.D ? a.d_q_weight : a.d_k_weight;  // (D is a multiple of 16: a CTA's columns are of one kind)
  if (out == nullptr) return;
  const float* rows = static_cast<const float*>(a.workspace) + d;
  float s = 0.0f;
#pragma unroll 8
  for (int64_t r = wid * 4 + (lane >> 3); r < p.cut.ctas; r += kSumThreads / 8) s += rows[r * 2 * a.D];
  s += __shfl_xor_sync(kAll, s, 8);
  s += __shfl_xor_sync(kAll, s, 16);
  if (lane < 8) part[wid][lane] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumThreads / 32; ++i) v += part[i][threadIdx.x];
    out[d - (d < a.D ? 0 : a.D) - (lane & 7) + threadIdx.x] = v;
  }
}

template <typename A, int G, int STYLE>
cudaError_t launch_forward(const HeadParams& p, cudaStream_t stream) {
  const int smem = kFwdThreads / 32 * (kSlotBytes<kFwdSlots, 2> + p.cut.cache_bytes);
  static_assert(kFwdThreads / 32 * (kSlotBytes<kFwdSlots, 2> + 32 * 256) <= 48 * 1024, "32 lanes' turns of both kinds fit without asking");
  return launch_pdl<HeadParams>(head_norm_kernel<A, G, STYLE>, dim3(static_cast<unsigned>(p.cut.ctas)), kFwdThreads, smem, p.a.flags & MFR_FLAG_PDL, stream, p);
}
template <typename A, int G, int STYLE>
cudaError_t launch_backward(const HeadParams& p, cudaStream_t stream) {
  static_assert(kSlotBytes<kBwdSlots, 4> >= 2 * MFR_MAX_HEAD_DIM * 4, "a warp's sums fit in its slots");
  const int smem = kBwdWarps * bwd_warp_bytes(p.cut.cache_bytes);
  const cudaError_t e = allow_smem<head_norm_grad_kernel<A, G, STYLE>>(kBwdWarps * bwd_warp_bytes(32 * 64));  // 32 lanes' turns
  if (e != cudaSuccess) return e;
  return launch_pdl<HeadParams>(head_norm_grad_kernel<A, G, STYLE>, dim3(static_cast<unsigned>(p.cut.ctas)), kBwdThreads, smem, p.a.flags & MFR_FLAG_PDL, stream, p);
}

template <typename A, int STYLE>
cudaError_t launch_g(const HeadParams& p, bool backward, cudaStream_t stream) {
  const int lanes = p.a.D / 16;
#define MFR_HEADS(G) \
  if (lanes <= G) return backward ? launch_backward<A, G, STYLE>(p, stream) : launch_forward<A, G, STYLE>(p, stream)
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
cudaError_t launch_s(const HeadParams& p, bool backward, cudaStream_t stream) {
  return p.a.style == MFR_ROTARY_HALF ? launch_g<A, MFR_ROTARY_HALF>(p, backward, stream)
                                      : launch_g<A, MFR_ROTARY_INTERLEAVED>(p, backward, stream);
}

int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Cuts the work: as many groups on a token as its larger kind has heads for.  `entry_bytes`: of a turn cache.
HeadCut cut_heads(int T, int q_heads, int k_heads, int D, int entry_bytes) {
  HeadCut c{};
  int G = 1;
  while (G < D / 16) G *= 2;
  const int groups = 32 / G, heads = std::max(q_heads, k_heads);
  while ((2 << c.gpt_log2) <= groups && (2 << c.gpt_log2) <= heads) ++c.gpt_log2;
  c.q_rounds = static_cast<int>(ceil_div64(q_heads, 1 << c.gpt_log2));
  c.k_rounds = static_cast<int>(ceil_div64(k_heads, 1 << c.gpt_log2));
  const int tokens = groups >> c.gpt_log2;
  c.cache_bytes = tokens * 4 * G * entry_bytes;
  c.blocks = ceil_div64(T, tokens);
  return c;
}

// Forward: a warp for each block, or as many as a block has rounds for when the blocks alone leave warps idle.
HeadCut cut_forward(int T, int q_heads, int k_heads, int D) {
  HeadCut c = cut_heads(T, q_heads, k_heads, D, 64);
  const int64_t fill = 152 * kFwdCtas * (kFwdThreads / 32);
  c.splits = static_cast<int>(std::min<int64_t>(c.q_rounds + c.k_rounds, std::max<int64_t>(1, fill / c.blocks)));
  c.warps = c.blocks * c.splits;
  c.ctas = ceil_div64(c.warps, kFwdThreads / 32);
  return c;
}

// Backward: the warps that the GPU holds, or one for each round.
HeadCut cut_backward(int T, int q_heads, int k_heads, int D) {
  HeadCut c = cut_heads(T, q_heads, k_heads, D, 16);
  c.warps = std::min<int64_t>(static_cast<int64_t>(kHeadGradBlocks) * kBwdWarps, c.blocks * (c.q_rounds + c.k_rounds));
  c.ctas = ceil_div64(c.warps, kBwdWarps);
  return c;
}

}  // namespace

int head_grad_rows(int T, int q_heads, int k_heads, int D) {
  return static_cast<int>(cut_backward(T, q_heads, k_heads, D).ctas);
}

cudaError_t launch_head_norm(const mfr_head_norm_args& a, cudaStream_t stream) {
  const HeadParams p{a, cut_forward(a.T, a.q_heads, a.k_heads, a.D)};
  if (p.cut.ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  return a.act_dtype == MFR_BF16 ? launch_s<__nv_bfloat16>(p, false, stream) : launch_s<__half>(p, false, stream);
}

cudaError_t launch_head_norm_backward(const mfr_head_norm_args& a, cudaStream_t stream) {
  const HeadParams p{a, cut_backward(a.T, a.q_heads, a.k_heads, a.D)};
  cudaError_t e = cudaSuccess;
  if (a.T > 0) e = a.act_dtype == MFR_BF16 ? launch_s<__nv_bfloat16>(p, true, stream) : launch_s<__half>(p, true, stream);
  // (no tokens: no partial sums, and the weight gradients are zeros)
  if (e != cudaSuccess || (a.d_q_weight == nullptr && a.d_k_weight == nullptr)) return e;
  return launch_pdl<HeadParams>(head_weight_grad_kernel, dim3(2 * a.D / 8), kSumThreads, 0, a.flags & MFR_FLAG_PDL, stream, p);
}

}  // namespace mfr
