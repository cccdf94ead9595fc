// Per-head RMSNorm of queries and keys and their position rotation in one pass, and its gradients.
//
// A group of G lanes (the power of two from D / 16 on) takes one head at a time; each of its first D / 16
// lanes holds 16 elements as two 16-byte vectors, chosen so that both elements of every rotated pair lie in
// the same lane:
//   half style         vectors p and p + rot/16 (elements i and i + rot/2), then the unrotated rest in twos
//   interleaved style  vectors 2p and 2p + 1 (neighbouring elements)
// so the rotation needs no exchange, and a head's sum of squares takes log2(G) shuffles.  A lane turns the
// same 8 pairs of every head of a token, so their sines and cosines are computed once a token and kept in
// registers.  Each warp walks a contiguous range of (token, head) items, its groups on neighbouring heads.
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

struct HeadParams {
  mfr_head_norm_args a;
  int64_t items;     // (token, head) pairs of this launch
  int64_t per_warp;  // items of one warp, a multiple of its groups
  int q_blocks;      // backward: CTAs [0, q_blocks) take the queries, the rest the keys
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
  int pair0;         // first pair (half: pairs pair0..pair0+7; interleaved: the same)
  int pairs;         // how many of the 8 are rotated
};

__device__ __forceinline__ LaneMap lane_map(int p, int rot, int style) {
  LaneMap m;
  m.pair0 = 8 * p;
  if (style == MFR_ROTARY_INTERLEAVED) {
    m.off_a = 16 * p;
    m.off_b = 16 * p + 8;
  } else if (16 * p < rot) {
    m.off_a = 8 * p;
    m.off_b = 8 * p + rot / 2;
  } else {
    m.off_a = 16 * p;  // rot + 16 (p - rot/16)
    m.off_b = 16 * p + 8;
  }
  m.pairs = min(8, max(0, rot / 2 - 8 * p));
  return m;
}

// Sines and cosines of a lane's pairs at a position, times rotary_scale; (1, 0) for unrotated pairs.
__device__ __forceinline__ void turns(const mfr_head_norm_args& a, const LaneMap& m, int64_t pos, float cs[8], float sn[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.0f;
    sn[i] = 0.0f;
    if (i < m.pairs) {
      const uint64_t u = turn_of(a.inv_freq[m.pair0 + i]) * static_cast<uint64_t>(pos);
      // the nearest 2^-32 turn, as a half turn in [-1, 1)
      const float h = static_cast<float>(static_cast<int32_t>((u + 0x80000000ULL) >> 32)) * 4.656612873077393e-10f;
      float s, c;
      sincospif(h, &s, &c);
      cs[i] = c * a.rotary_scale;
      sn[i] = s * a.rotary_scale;
    }
  }
}

__device__ __forceinline__ int64_t position_of(const mfr_head_norm_args& a, int64_t t) {
  return (a.flags & MFR_FLAG_POSITIONS_64) ? static_cast<const int64_t*>(a.positions)[t]
                                           : static_cast<const int32_t*>(a.positions)[t];
}

template <typename A>
__device__ __forceinline__ void load16(const uint8_t* base, int off_a, int off_b, bool on, float v[16]) {
  unpack8<A>(on ? ldg16(base + 2 * off_a) : make_uint4(0, 0, 0, 0), v);
  unpack8<A>(on ? ldg16(base + 2 * off_b) : make_uint4(0, 0, 0, 0), v + 8);
}

template <typename A>
__device__ __forceinline__ void store16(uint8_t* base, int off_a, int off_b, const float v[16]) {
  *reinterpret_cast<uint4*>(base + 2 * off_a) =
      make_uint4(Act<A>::pack(v[0], v[1]), Act<A>::pack(v[2], v[3]), Act<A>::pack(v[4], v[5]), Act<A>::pack(v[6], v[7]));
  *reinterpret_cast<uint4*>(base + 2 * off_b) =
      make_uint4(Act<A>::pack(v[8], v[9]), Act<A>::pack(v[10], v[11]), Act<A>::pack(v[12], v[13]), Act<A>::pack(v[14], v[15]));
}

// A kind's weight at a lane's elements (ones without a weight).
template <typename A>
__device__ __forceinline__ void load_weight(const void* w, const LaneMap& m, bool on, float v[16]) {
  if (w != nullptr) {
    load16<A>(static_cast<const uint8_t*>(w), m.off_a, m.off_b, on, v);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 1.0f;
  }
}

// Turns a lane's pairs by +angle (sign 1) or back (sign -1).
template <int STYLE>
__device__ __forceinline__ void turn_pairs(float v[16], const float cs[8], const float sn[8], float sign) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x = STYLE == MFR_ROTARY_HALF ? v[i] : v[2 * i];
    float& y = STYLE == MFR_ROTARY_HALF ? v[i + 8] : v[2 * i + 1];
    const float s = sign * sn[i];
    const float u = x * cs[i] - y * s;
    y = y * cs[i] + x * s;
    x = u;
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ uint8_t* head_row(const mfr_heads& h, int64_t t, int head) {
  return static_cast<uint8_t*>(h.data) + 2 * (t * h.token_stride + head * h.head_stride);
}

template <typename A, int G, int STYLE>
__global__ void __launch_bounds__(kHeadThreads) head_norm_kernel(const __grid_constant__ HeadParams p) {
  const mfr_head_norm_args& a = p.a;
  const int lane = threadIdx.x & 31, group = lane / G, groups = 32 / G;
  const bool on = lane % G < a.D / 16;
  const LaneMap m = lane_map(lane % G, a.rot, STYLE);
  const int heads = a.q_heads + a.k_heads;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kHeadWarps + (threadIdx.x >> 5);
  const int64_t first = warp * p.per_warp;
  const int64_t end = first + p.per_warp < p.items ? first + p.per_warp : p.items;
  pdl_launch_dependents();
  pdl_wait();
  int64_t t_now = -1, pos = -1;
  int kind_now = -1;
  float cs[8], sn[8], w[16];
  int64_t t = first / heads;
  int h = static_cast<int>(first % heads) + group;
  for (int64_t i = first; i < end; i += groups, h += groups) {  // the same trip count for all lanes
    while (h >= heads) {
      h -= heads;
      ++t;
    }
    const bool live = on && i + group < end;
    float x[16];
    const int kind = h < a.q_heads ? 0 : 1;
    const mfr_heads& in = kind == 0 ? a.q : a.k;
    const mfr_heads& out = kind == 0 ? a.q_out : a.k_out;
    const int hh = kind == 0 ? h : h - a.q_heads;
    if (live && t != t_now) {
      t_now = t;
      pos = position_of(a, t);
      if (pos >= 0) turns(a, m, pos, cs, sn);
    }
    if (live && kind != kind_now) {
      kind_now = kind;
      load_weight<A>(kind == 0 ? a.q_weight : a.k_weight, m, true, w);
    }
    const bool work = live && pos >= 0;
    load16<A>(work ? head_row(in, t, hh) : nullptr, m.off_a, m.off_b, work, x);
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) sq = __fmaf_rn(x[j], x[j], sq);
    sq = group_sum<G>(sq);
    if (work) {
      const float r = rms_rstd(sq, a.D, a.eps);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = x[j] * r * w[j];
      turn_pairs<STYLE>(x, cs, sn, 1.0f);
      store16<A>(head_row(out, t, hh), m.off_a, m.off_b, x);
    } else if (live && (a.flags & MFR_FLAG_ZERO_PADDING)) {
      store16<A>(head_row(out, t, hh), m.off_a, m.off_b, x);  // zeros
    }
  }
}

// Gradient.  CTAs [0, q_blocks) walk the queries, the rest the keys; each keeps its lanes' share of the
// weight gradient in registers and leaves one row of partial sums in the workspace.
template <typename A, int G, int STYLE>
__global__ void __launch_bounds__(kHeadThreads) head_norm_grad_kernel(const __grid_constant__ HeadParams p) {
  extern __shared__ float part[];  // [kHeadWarps][D]
  const mfr_head_norm_args& a = p.a;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = lane / G, groups = 32 / G;
  const bool on = lane % G < a.D / 16;
  const LaneMap m = lane_map(lane % G, a.rot, STYLE);
  const bool keys = static_cast<int>(blockIdx.x) >= p.q_blocks;
  const int block = keys ? blockIdx.x - p.q_blocks : blockIdx.x;
  const int blocks = keys ? gridDim.x - p.q_blocks : p.q_blocks;
  const int heads = keys ? a.k_heads : a.q_heads;
  const mfr_heads& in = keys ? a.k : a.q;
  const mfr_heads& out = keys ? a.k_out : a.q_out;
  const mfr_heads& dout = keys ? a.d_k_out : a.d_q_out;
  const bool want = (keys ? a.d_k_weight : a.d_q_weight) != nullptr;
  // contiguous items a warp, in whole rounds of its groups
  const int64_t items = static_cast<int64_t>(a.T) * heads;
  const int64_t rounds = (items + groups - 1) / groups;
  const int64_t warps = static_cast<int64_t>(blocks) * kHeadWarps, me = static_cast<int64_t>(block) * kHeadWarps + wid;
  const int64_t first = rounds * me / warps * groups;
  int64_t end = rounds * (me + 1) / warps * groups;
  end = end < items ? end : items;
  pdl_launch_dependents();
  pdl_wait();
  float w[16], dw[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) dw[j] = 0.0f;
  load_weight<A>(keys ? a.k_weight : a.q_weight, m, on, w);
  int64_t t_now = -1, pos = -1;
  float cs[8], sn[8];
  int64_t t = first / heads;
  int h = static_cast<int>(first % heads) + group;
  for (int64_t i = first; i < end; i += groups, h += groups) {
    while (h >= heads) {
      h -= heads;
      ++t;
    }
    const bool live = on && i + group < end;
    if (live && t != t_now) {
      t_now = t;
      pos = position_of(a, t);
      if (pos >= 0) turns(a, m, pos, cs, sn);
    }
    const bool work = live && pos >= 0;
    float x[16], g[16];
    load16<A>(work ? head_row(in, t, h) : nullptr, m.off_a, m.off_b, work, x);
    load16<A>(work ? head_row(dout, t, h) : nullptr, m.off_a, m.off_b, work, g);
    if (work) turn_pairs<STYLE>(g, cs, sn, -1.0f);
    float sq = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      sq = __fmaf_rn(x[j], x[j], sq);
      dot = __fmaf_rn(g[j] * w[j], x[j], dot);
    }
    sq = group_sum<G>(sq);
    dot = group_sum<G>(dot);
    if (work) {
      const float r = rms_rstd(sq, a.D, a.eps);
      const float c = __fdiv_rn(dot, static_cast<float>(a.D)) * r * r;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        dw[j] = __fmaf_rn(g[j] * r, x[j], dw[j]);
        x[j] = r * (g[j] * w[j] - x[j] * c);
      }
    }
    if (live) store16<A>(head_row(out, t, h), m.off_a, m.off_b, x);  // zeros for a padding token
  }
  if (!want) return;
  // over the warp's groups (lanes G apart), then over the CTA's warps in order
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int o = 16; o >= G; o >>= 1) dw[j] += __shfl_xor_sync(kAll, dw[j], o);
  }
  if (group == 0 && on) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      part[wid * a.D + m.off_a + j] = dw[j];
      part[wid * a.D + m.off_b + j] = dw[j + 8];
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
  const int64_t b0 = keys ? p.q_blocks : 0, b1 = keys ? p.items : p.q_blocks;  // items: the gradient kernel's CTAs
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

}  // namespace

cudaError_t launch_head_norm(const mfr_head_norm_args& a, cudaStream_t stream) {
  HeadParams p{a, 0, 0, 0};
  const int groups = groups_of(a.D), heads = a.q_heads + a.k_heads;
  p.items = static_cast<int64_t>(a.T) * heads;
  // A token's heads a warp when that gives every SM its warps, else fewer, down to one round of the groups.
  const int64_t rounds = (p.items + groups - 1) / groups;
  int64_t per = (heads + groups - 1) / groups;
  const int64_t fill = (rounds + 152 * 24 - 1) / (152 * 24);  // rounds a warp at 24 warps an SM
  if (per > fill) per = fill;
  p.per_warp = per * groups;
  const int64_t warps = (rounds + per - 1) / per;
  const int64_t blocks = (warps + kHeadWarps - 1) / kHeadWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return a.act_dtype == MFR_BF16 ? launch_s<__nv_bfloat16>(p, static_cast<int>(blocks), false, stream)
                                 : launch_s<__half>(p, static_cast<int>(blocks), false, stream);
}

cudaError_t launch_head_norm_backward(const mfr_head_norm_args& a, cudaStream_t stream) {
  HeadParams p{a, 0, 0, 0};
  const int groups = groups_of(a.D);
  // CTAs in proportion to the heads of each kind, at least one where there are any
  const int64_t warps = (static_cast<int64_t>(a.T) * (a.q_heads + a.k_heads) + groups - 1) / groups;
  int64_t blocks = (warps + kHeadWarps - 1) / kHeadWarps;
  if (blocks > kHeadGradBlocks) blocks = kHeadGradBlocks;
  if (blocks < 2) blocks = 2;
  int q = static_cast<int>(blocks * a.q_heads / (a.q_heads + a.k_heads));
  if (a.q_heads > 0 && q == 0) q = 1;
  if (a.k_heads > 0 && q == blocks) q = static_cast<int>(blocks) - 1;
  p.q_blocks = q;
  p.items = blocks;
  cudaError_t e = cudaSuccess;
  if (a.T == 0) {
    p.q_blocks = 0;
    p.items = 0;  // no partial sums: the weight gradients are zeros
  } else {
    e = a.act_dtype == MFR_BF16 ? launch_s<__nv_bfloat16>(p, static_cast<int>(blocks), true, stream)
                                : launch_s<__half>(p, static_cast<int>(blocks), true, stream);
  }
  if (e != cudaSuccess || (a.d_q_weight == nullptr && a.d_k_weight == nullptr)) return e;
  return launch_pdl<HeadParams>(head_weight_grad_kernel, dim3(2 * ((a.D + 31) / 32)), kSumThreads, 0, a.flags & MFR_FLAG_PDL, stream, p);
}

}  // namespace mfr
