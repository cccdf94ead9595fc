// Routing to experts: scores, expert groups, the K best experts of each token, their weights, and the
// expert order of the routes; and the gradient of the weights to the logits.
//
// One warp takes one token.  Lane l holds the NV consecutive experts from l * NV on, so among equal scores
// the lowest lane, and within it the lowest slot, is the lowest expert index.
//
// The order of the chosen experts is that of 64-bit choice scores.  Without a bias a score orders as its
// logit, and the logits are compared as they are.  With a bias (and for group scores that are sums) the
// scores are computed in FP32 with a bound on the error of each, from its own size (near_of, slack_of).  Where the
// ranges of two neighbours in the order meet, or those of a kept and a dropped group, what lies there is decided
// again in FP64: the groups and candidates concerned, or, where they are many, all experts (slow_choice).  Random
// inputs need that about once in a thousand tokens.
//
// The expert order is a stable counting sort.  A CTA takes a contiguous chunk of tokens and marks each
// route in a bitmap [expert][token of the segment]: a route's rank among its expert's routes is the number
// of marks below its own, so the marks may be set in any order (atomicOr) with the same result.  Small batches
// run as one cluster whose CTAs read each other's counts from shared memory, in one launch; larger ones leave
// the chunks' counts in the workspace, and a second kernel (order_kernel) adds those of the chunks before its own.
//
// Bound by instructions, not by HBM: a token of 256 experts takes about 430 warp instructions for a choice by logits
// and about 1000 with a bias, groups, 64-bit decisions and the order's marks, while its logits take 0.15 ns of HBM time.
// Ranking the few candidates by counting is what keeps it there: one expert after the other took 1835.  Measured on
// GB300, in a graph: 16384 tokens of 256 experts, top-8, 9.3 us by logits and 19.8 us with bias and groups (the logits
// are 2.5 us at the copy bandwidth; 28.5 us with 2 of 8 groups kept, whose 64 experts are all candidates), and 7 us more
// for the order; one token 2.5 us, 3.8 us with the order.
#include "layer_launch.h"

namespace mfr {
namespace {

constexpr float kInf = __builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSegTokens = 128;            // tokens whose routes are ranked together
constexpr int kSegWords = kSegTokens / 32;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float fast_exp2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
__device__ __forceinline__ float fast_rcp(float t) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// A launch: the call's arguments, and what every token would otherwise divide for.
struct RouteParams {
  mfr_route_args a;
  int group_size;   // experts of a group
  int width_log2;   // a group is 2^width_log2 whole lanes, aligned; -1: it is not
  int clustered;    // the whole batch runs as one cluster
  int chunk, extra; // chunk b holds `chunk` tokens, and one more for b < extra
};

// A float as an unsigned integer of the same order (no NaN, no -0).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ (static_cast<uint32_t>(static_cast<int32_t>(~u) >> 31) | 0x80000000u));
}
__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(kAll, ordered(v))); }

__device__ __forceinline__ double unordered64(int64_t u) {
  return __longlong_as_double(u ^ (static_cast<int64_t>(static_cast<uint64_t>(u >> 63) >> 1)));
}

// A logit or weight of any of the three types, as FP32.
__device__ __forceinline__ float load_any(const void* base, int64_t i, int dtype) {
  if (dtype == MFR_FP32) return static_cast<const float*>(base)[i];
  const uint16_t b = static_cast<const uint16_t*>(base)[i];
  return dtype == MFR_BF16 ? __uint_as_float(static_cast<uint32_t>(b) << 16) : __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ void store_any(void* base, int64_t i, int dtype, float v) {
  if (dtype == MFR_FP32)
    static_cast<float*>(base)[i] = v;
  else if (dtype == MFR_BF16)
    static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(base)[i] = __float2half_rn(v);
}

// NaN becomes -inf: such an expert cannot be taken.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -kInf); }

// A double as an integer of the same order (no NaN; -0 becomes +0): comparing doubles is as slow as adding them.
__device__ __forceinline__ int64_t ordered64(double v) {
  const int64_t b = __double_as_longlong(v + 0.0);
  return b ^ (static_cast<int64_t>(static_cast<uint64_t>(b >> 63) >> 1));
}

// NV logits of one lane, in vectors when all of them exist and the address allows.
template <typename L, int NV>
__device__ __forceinline__ void load_logits(const L* row, int e0, int E, float x[NV]) {
  constexpr int kBytes = NV * static_cast<int>(sizeof(L));
  constexpr int kVec = kBytes >= 16 ? 16 : kBytes;
  const L* p = row + e0;
  if constexpr (kVec >= 4) {
    if (e0 + NV <= E && (reinterpret_cast<uintptr_t>(p) & (kVec - 1)) == 0) {
      uint32_t raw[kBytes / 4];
      if constexpr (kVec == 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
          const uint4 v = reinterpret_cast<const uint4*>(p)[i];
          raw[4 * i] = v.x;
          raw[4 * i + 1] = v.y;
          raw[4 * i + 2] = v.z;
          raw[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) raw[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if constexpr (sizeof(L) == 4) {
          x[j] = __uint_as_float(raw[j]);
        } else {
          const float2 f = Act<L>::unpack(raw[j / 2]);
          x[j] = j % 2 ? f.y : f.x;
        }
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) x[j] = clean(x[j]);
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v = -kInf;
    if (e0 + j < E) {
      if constexpr (sizeof(L) == 4)
        v = p[j];
      else
        v = static_cast<float>(p[j]);
    }
    x[j] = clean(v);
  }
}

// NV consecutive floats of a lane in shared memory, in vectors (a lane's share is 4 NV bytes, aligned to that).
template <int NV>
__device__ __forceinline__ void store_lane(float* base, int lane, const float (&v)[NV]) {
  if constexpr (NV >= 4) {
#pragma unroll
    for (int j = 0; j < NV; j += 4) reinterpret_cast<float4*>(base + lane * NV)[j / 4] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) base[lane * NV + j] = v[j];
  }
}
template <int NV>
__device__ __forceinline__ void load_lane(const float* base, int lane, float (&v)[NV]) {
  if constexpr (NV >= 4) {
#pragma unroll
    for (int j = 0; j < NV; j += 4) {
      const float4 f = reinterpret_cast<const float4*>(base + lane * NV)[j / 4];
      v[j] = f.x, v[j + 1] = f.y, v[j + 2] = f.z, v[j + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = base[lane * NV + j];
  }
}

// The two best of two pairs of best values.
template <typename F>
__device__ __forceinline__ void merge_top2(F& a, F& b, F a2, F b2) {
  const F lo = a < a2 ? a : a2;
  const F hi = b > b2 ? b : b2;
  a = a > a2 ? a : a2;
  b = lo > hi ? lo : hi;
}

// How far apart two FP32 choice scores must lie for their order to be that of the exact ones: each holds a score that is
// `err` off and the rounding of its bias's addition, 2^-24 of it (twice that here).
__device__ __forceinline__ float near_of(float err, float v, float w) { return __fmaf_rn(1.2e-7f, fabsf(v) + fabsf(w), 2.0f * err); }

// The FP32 group score of a group's two best choice scores (-inf: none).  A sum that leaves FP32 stays at its ends: it is
// finite in 64 bits, so the group can be kept, and the error bound sends what lies near to 64 bits.
__device__ __forceinline__ float group_score(float best, float second, bool top2) {
  return top2 && second > -kInf ? fminf(fmaxf(best + second, -3.402823466e38f), 3.402823466e38f) : best;
}

// ---------------------------------------------------------------------------------------------------
// The choice again, in 64 bits
// ---------------------------------------------------------------------------------------------------

// A logit's score before the softmax's division, in FP64.
__device__ __forceinline__ double raw_score64(int score, double x, double top) {
  if (!(x > -kInf)) return 0.0;
  if (score == MFR_SCORE_SOFTMAX) return x == top ? 1.0 : exp(x - top);
  return 1.0 / (1.0 + exp(-x));
}

// The softmax's sum over the token's logits, in FP64 (1 for the sigmoid).
template <typename L>
__device__ __noinline__ double score_sum64(const mfr_route_args& a, const L* row, int lane, double top) {
  if (a.score != MFR_SCORE_SOFTMAX) return 1.0;
  double sum = 0.0;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) sum += raw_score64(a.score, clean(static_cast<float>(row[e])), top);
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  return sum;
}

// Chooses the token's experts with every score in FP64 (local arrays: this path is rare).  Lane l gets the
// ids of places l and l + 32.  (Out of line, and by value: what the hot path keeps in registers must not have an address.)
template <typename L, int NV>
__device__ __noinline__ int2 slow_choice(const mfr_route_args& a, const L* row, int lane) {
  constexpr int64_t kNone = INT64_MIN;
  int64_t c[NV];  // choice scores, as ordered integers
  double s[NV];
  const int e0 = lane * NV;
  float top = -kInf;
#pragma unroll 1
  for (int j = 0; j < NV; ++j)
    if (e0 + j < a.E) top = fmaxf(top, clean(static_cast<float>(row[e0 + j])));
  top = warp_max(top);
  const double inv = 1.0 / score_sum64(a, row, lane, top);
#pragma unroll 1
  for (int j = 0; j < NV; ++j) {
    c[j] = kNone;
    s[j] = 0.0;
    if (e0 + j >= a.E) continue;
    const float x = clean(static_cast<float>(row[e0 + j]));
    if (!(x > -kInf)) continue;
    s[j] = raw_score64(a.score, x, top) * inv;
    const double v = a.bias != nullptr ? s[j] + static_cast<double>(a.bias[e0 + j]) : static_cast<double>(x);
    if (v > -kInf) c[j] = ordered64(v);
  }
  if (a.num_groups > 1) {
    const bool top2 = a.group_score == MFR_GROUP_TOP2;
    const int size = a.E / a.num_groups;
    int64_t mine = kNone;  // lane g: group g's score
    for (int g = 0; g < a.num_groups; ++g) {
      int64_t b1 = kNone, b2 = kNone;
#pragma unroll 1
      for (int j = 0; j < NV; ++j) {
        const int e = e0 + j;
        if (e < a.E && e / size == g && c[j] != kNone)
          merge_top2(b1, b2, top2 && a.bias == nullptr ? ordered64(s[j]) : c[j], kNone);
      }
      for (int o = 16; o > 0; o >>= 1) {
        const int64_t v1 = __shfl_xor_sync(kAll, b1, o), v2 = __shfl_xor_sync(kAll, b2, o);
        merge_top2(b1, b2, v1, v2);
      }
      if (top2 && b2 != kNone) b1 = ordered64(unordered64(b1) + unordered64(b2));
      if (lane == g) mine = b1;
    }
    int rank = 0;
    for (int g = 0; g < a.num_groups; ++g) {
      const int64_t v = __shfl_sync(kAll, mine, g);
      rank += (v > mine || (v == mine && g < lane)) ? 1 : 0;
    }
    const unsigned kept = __ballot_sync(kAll, lane < a.num_groups && rank < a.topk_groups && mine != kNone);
#pragma unroll 1
    for (int j = 0; j < NV; ++j)
      if (e0 + j < a.E && !((kept >> ((e0 + j) / size)) & 1)) c[j] = kNone;
  }
  int id0 = -1, id1 = -1;
  for (int k = 0; k < a.K; ++k) {
    int64_t best = kNone;
    int at = INT32_MAX;
#pragma unroll 1
    for (int j = 0; j < NV; ++j)
      if (c[j] > best) {
        best = c[j];
        at = e0 + j;
      }
    for (int o = 16; o > 0; o >>= 1) {
      const int64_t v = __shfl_xor_sync(kAll, best, o);
      const int i = __shfl_xor_sync(kAll, at, o);
      if (v > best || (v == best && i < at)) {
        best = v;
        at = i;
      }
    }
    if (at == INT32_MAX) break;
    if (at / NV == lane) c[at % NV] = kNone;
    if (lane == (k & 31)) (k < 32 ? id0 : id1) = at;
  }
  return make_int2(id0, id1);
}

// ---------------------------------------------------------------------------------------------------
// One token
// ---------------------------------------------------------------------------------------------------

constexpr int kList = 64;  // candidates that a warp can rank, two a lane

// A warp's shared memory: its token's choice scores, and the candidates' scores, experts and 64-bit scores.
struct Scratch {
  float* scores;   // [32 * NV]
  int64_t* wide;   // [kList]
  float* value;    // [kList]
  int* expert;     // [kList]
};
template <int NV>
constexpr int kScratchBytes = 32 * NV * 4 + kList * 16;
template <int NV>
__device__ __forceinline__ Scratch scratch_of(uint8_t* base) {
  Scratch s;
  s.scores = reinterpret_cast<float*>(base);
  s.wide = reinterpret_cast<int64_t*>(base + 32 * NV * 4);
  s.value = reinterpret_cast<float*>(base + 32 * NV * 4 + kList * 8);
  s.expert = reinterpret_cast<int*>(base + 32 * NV * 4 + kList * 12);
  return s;
}

// The groups whose scores may lie on either side of the border between kept and dropped ones, decided again in FP64:
// kept ones that may be as low as the highest a dropped one may be (`highest_out`), and dropped ones that may be as high
// as the lowest a kept one may be (`lowest_in`).  sc.scores holds the values that the groups compare, lane g group g's
// score, its error bound `slack` and its second best value; `in`: whether it is kept.  Returns the groups kept, or 0 when
// too many values matter.
template <typename L, int NV>
__device__ __noinline__ unsigned decide_groups(const RouteParams& p, const L* row, int lane, uint8_t* scratch, float top, float mine,
                                               float second, float slack, bool in, float lowest_in, float highest_out) {
  const Scratch sc = scratch_of<NV>(scratch);
  const mfr_route_args& a = p.a;
  const bool top2 = a.group_score == MFR_GROUP_TOP2, biased = a.bias != nullptr;
  const bool here = lane < a.num_groups && mine > -kInf;
  const unsigned kept = __ballot_sync(kAll, in);
  const unsigned band = __ballot_sync(kAll, here && !(in ? mine - slack > highest_out : lowest_in > mine + slack));
  // the values that may be among a group's two best
  int n = 0, begin = 0, end = 0;
  for (unsigned m = band; m; m &= m - 1) {
    const int g = __ffs(m) - 1;
    const float least = fmaxf(__shfl_sync(kAll, (top2 ? second : mine) - 2.0f * slack, g), -3.402823466e38f);
    if (lane == g) begin = n;
    for (int i0 = 0; i0 < p.group_size; i0 += 32) {
      const int i = i0 + lane;
      const bool take = i < p.group_size && sc.scores[g * p.group_size + i] >= least;
      const unsigned votes = __ballot_sync(kAll, take);
      const int at = n + __popc(votes & ((1u << lane) - 1));
      if (take && at < kList) sc.expert[at] = g * p.group_size + i;
      n += __popc(votes);
      if (n > kList) return 0;
    }
    if (lane == g) end = n;
  }
  __syncwarp();
  const double inv = 1.0 / score_sum64(a, row, lane, top);
  for (int q = lane; q < n; q += 32) {
    const int e = sc.expert[q];
    const double v = raw_score64(a.score, clean(static_cast<float>(row[e])), top) * inv;
    sc.wide[q] = ordered64(biased ? v + static_cast<double>(a.bias[e]) : v);
  }
  __syncwarp();
  int64_t score = INT64_MIN;
  if ((band >> lane) & 1) {
    int64_t b1 = INT64_MIN, b2 = INT64_MIN;
    for (int q = begin; q < end; ++q) merge_top2(b1, b2, sc.wide[q], static_cast<int64_t>(INT64_MIN));
    score = top2 && b2 != INT64_MIN ? ordered64(unordered64(b1) + unordered64(b2)) : b1;
  }
  int rank = 0;
  for (unsigned m = band; m; m &= m - 1) {
    const int g = __ffs(m) - 1;
    const int64_t v = __shfl_sync(kAll, score, g);
    rank += (v > score || (v == score && g < lane)) ? 1 : 0;
  }
  const unsigned again = __ballot_sync(kAll, ((band >> lane) & 1) && rank < __popc(kept & band));
  __syncwarp();
  return (kept & ~band) | again;
}

// The candidates' ranks again, in FP64.
template <typename L, int NV>
__device__ __noinline__ int2 decide_candidates(const mfr_route_args& a, const L* row, int lane, uint8_t* scratch, float top, int n) {
  const Scratch sc = scratch_of<NV>(scratch);
  const double inv = 1.0 / score_sum64(a, row, lane, top);
  for (int q = lane; q < n; q += 32) {
    const int e = sc.expert[q];
    sc.wide[q] = ordered64(raw_score64(a.score, clean(static_cast<float>(row[e])), top) * inv + static_cast<double>(a.bias[e]));
  }
  __syncwarp();
  const int64_t v0 = lane < n ? sc.wide[lane] : 0, v1 = lane + 32 < n ? sc.wide[lane + 32] : 0;
  int rank0 = 0, rank1 = 0;
  for (int q = 0; q < n; ++q) {
    const int64_t u = sc.wide[q];
    rank0 += (u > v0 || (u == v0 && q < lane)) ? 1 : 0;
    rank1 += (u > v1 || (u == v1 && q < lane + 32)) ? 1 : 0;
  }
  return make_int2(rank0, rank1);
}

// Chooses and weighs the experts of one token whose logits are x.  Each lane gets up to two of them: the
// expert id[i] at place[i] of the token's list, or id -1; `taken` in all.  `bias`: the experts' biases in shared memory.  GENERAL:
// there are biases or groups; without them the logits decide and no score is needed for the choice.
template <typename L, int NV, bool GENERAL>
__device__ __forceinline__ void route_token(const RouteParams& p, int64_t t, float (&x)[NV], int lane, const float* bias,
                                            uint8_t* scratch, int (&id)[2], int (&place)[2], int& taken) {
  const Scratch sc = scratch_of<NV>(scratch);
  const mfr_route_args& a = p.a;
  const L* row = static_cast<const L*>(a.logits) + t * a.logits_stride;
  const int e0 = lane * NV;
  const bool softmax = a.score == MFR_SCORE_SOFTMAX;
  const bool top2 = GENERAL && a.num_groups > 1 && a.group_score == MFR_GROUP_TOP2;
  const bool biased = GENERAL && a.bias != nullptr;
  float (&c)[NV] = x;  // the logits become the choice scores

  float top = -kInf, inv = 0.0f;  // the largest logit, and 1 / the softmax's sum
  float err = 0.0f;               // how far an FP32 score may be from the exact one
  float s[NV];
  if (biased || top2 || (softmax && !a.renormalize)) {
    if (softmax) {
      float m = x[0];
#pragma unroll
      for (int j = 1; j < NV; ++j) m = fmaxf(m, x[j]);
      top = warp_max(m);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        s[j] = x[j] == top ? 1.0f : fast_exp2((x[j] - top) * kLog2e);
        if (!(x[j] > -kInf)) s[j] = 0.0f;
        sum += s[j];
      }
      sum = warp_sum(sum);
      inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) s[j] *= inv;
      // With d the distance to the top: ex2.approx is 2^-22 off and its argument d 1.35e-7, together 2.9e-7 of
      // the top's term at most (e^-d d <= 0.37); the sum by the mean of d, ln(E) at most, times 1.35e-7, 2^-22
      // and (NV + 5) 2^-24: 3.4e-6 relative; two roundings.  Below 4e-6 of the top's score.
      err = 4e-6f * inv;
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) s[j] = fast_rcp(1.0f + fast_exp2(-x[j] * kLog2e));  // 0 for -inf
      // s (1 - s) (2^-22 + |x| 7.5e-8) + s 2^-24 + s 2^-23, with s (1 - s) |x| <= 0.28: below 2.7e-7
      err = 2.7e-7f;
    }
  }
  if (biased) {
    float b[NV];
    load_lane<NV>(bias, lane, b);
#pragma unroll
    for (int j = 0; j < NV; ++j) c[j] = x[j] > -kInf ? clean(s[j] + b[j]) : -kInf;
  }

  bool close = false;  // a decision lies within the error bound and too many experts with it: all in FP64
  if (GENERAL && a.num_groups > 1) {
    const bool sums = top2 && !biased;  // groups compare sums of scores, experts compare logits
    // what the groups compare of the lane's experts, for the paths that read it from shared memory
    auto share_values = [&]() {
      float v[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = sums ? (c[j] > -kInf ? s[j] : -kInf) : c[j];
      store_lane<NV>(sc.scores, lane, v);
      __syncwarp();
    };
    float mine = -kInf, second = -kInf;  // a group's score and second best value: its lanes hold them, or lane g group g's
    // How far a group's FP32 score may be from the exact one: each value it adds is `err` off and has the rounding of its
    // bias's addition, 2^-24 of that value (and not of the sum, where the two cancel); the rest is for the sum's rounding
    // and for that of the comparisons.
    float slack = 0.0f;
    auto slack_of = [&](float best, float second) {
      const float size = top2 && second > -kInf ? fabsf(best) + fabsf(second) : fabsf(best);
      return (top2 ? 2.0f : 1.0f) * err + 2.4e-7f * fminf(size, 3.402823466e38f);
    };
    bool on = false;                     // the lane's group is kept, or group `lane` is
    const int w = p.width_log2;
    if (w >= 0) {
      if (sums) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float v = c[j] > -kInf ? s[j] : -kInf;
          second = fmaxf(second, fminf(mine, v));
          mine = fmaxf(mine, v);
        }
      } else if (top2) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          second = fmaxf(second, fminf(mine, c[j]));
          mine = fmaxf(mine, c[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) mine = fmaxf(mine, c[j]);
      }
      for (int o = (1 << w) >> 1; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(kAll, mine, o);
        if (top2) second = fmaxf(fminf(mine, m2), fmaxf(second, __shfl_xor_sync(kAll, second, o)));
        mine = fmaxf(mine, m2);
      }
      slack = slack_of(mine, second);
      if (top2) mine = group_score(mine, second, true);
      // the best group again and again; among equal ones the lowest lane's
      const uint32_t key = ordered(mine + 0.0f);
      const uint32_t none = ordered(-kInf);
      for (int i = 0; i < a.topk_groups; ++i) {
        const uint32_t m = __reduce_max_sync(kAll, on ? 0 : key);
        if (m <= none) break;
        const int first = __ffs(__ballot_sync(kAll, !on && key == m)) - 1;
        on = on || (lane >> w) == (first >> w);
      }
    } else {
      share_values();
      if (lane < a.num_groups) {
        for (int i = 0; i < p.group_size; ++i) {
          const float v = sc.scores[lane * p.group_size + i];
          second = fmaxf(second, fminf(mine, v));
          mine = fmaxf(mine, v);
        }
        slack = slack_of(mine, second);
        mine = group_score(mine, second, top2);
      }
      __syncwarp();
      int rank = 0;
      for (int g = 0; g < a.num_groups; ++g) {
        const float v = __shfl_sync(kAll, mine, g);
        rank += (v > mine || (v == mine && g < lane)) ? 1 : 0;
      }
      on = rank < a.topk_groups && mine > -kInf;
    }
    unsigned kept = 0;  // by group
    bool by_group = w < 0;
    if (top2 || biased) {
      const float lowest_in = -warp_max(on ? slack - mine : -kInf), highest_out = warp_max(on ? -kInf : mine + slack);
      if (__any_sync(kAll, highest_out > -kInf && !(lowest_in > highest_out))) {  // (the same for all lanes)
        if (w >= 0) {
          // group g's to lane g
          const int from = (lane << w) & 31;
          mine = __shfl_sync(kAll, mine, from);
          second = __shfl_sync(kAll, second, from);
          slack = __shfl_sync(kAll, slack, from);
          on = __shfl_sync(kAll, on, from);
          if (lane >= a.num_groups) {
            mine = -kInf;
            on = false;
          }
          share_values();
        }
        kept = decide_groups<L, NV>(p, row, lane, scratch, top, mine, second, slack, on, lowest_in, highest_out);
        close = kept == 0;
        if (w >= 0) on = (kept >> (lane >> w)) & 1;
        by_group = false;
      }
    }
    if (w >= 0) {
      if (!on) {
#pragma unroll
        for (int j = 0; j < NV; ++j) c[j] = -kInf;
      }
    } else {
      if (by_group) kept = __ballot_sync(kAll, on);
      int g = e0 / p.group_size, left = p.group_size - e0 % p.group_size;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!((kept >> (g & 31)) & 1)) c[j] = -kInf;
        if (--left == 0) {
          left = p.group_size;
          ++g;
        }
      }
    }
  }

  id[0] = id[1] = -1;
  place[0] = lane;
  place[1] = lane + 32;
  int n = kList + 1;                // candidates
  float z[2] = {-kInf, -kInf};      // their scores: without a bias, their logits
  bool reload = biased;
  if (!close && a.K < kList) {
    // Every expert from some score on is a candidate, and the candidates are ranked by counting.  The K + 1 best of
    // the lanes' best bound the K + 1 best experts from below (about 10 candidates of 256 for K = 8).
    float best = c[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) best = fmaxf(best, c[j]);
    uint32_t key = ordered(best);
    const uint32_t first = __reduce_max_sync(kAll, key);
    uint32_t tau = first;
    if (a.K < 32) {
#pragma unroll 8
      for (int k = 0; k < a.K; ++k) {
        if (key == tau) key = 0;
        tau = __reduce_max_sync(kAll, key);
      }
    } else {
      tau = 0;
    }
    const float most = unordered(first);
    // fewer lanes than that have any: all experts that can be taken are candidates
    constexpr float kLowest = -3.402823466e38f;
    float least = tau > ordered(-kInf) ? unordered(tau) : kLowest;
    // An expert just below that one may come before it in 64 bits: with a bias the cut lies clear of the K-th best by
    // near_of and a little for this subtraction's rounding.
    if (biased) least = fmaxf(least - __fmaf_rn(3.6e-7f, fabsf(least), 2.5f * err), kLowest);
    bool bisected = false;
    unsigned mask = 0;
    auto select = [&]() {
      mask = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) mask |= c[j] >= least ? 1u << j : 0u;
      return __popc(mask);
    };
    // the candidates up to and with the lane's own
    auto scan = [&](int own) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, own, o);
        if (lane >= o) own += v;
      }
      return own;
    };
    int before = select();
    n = __reduce_add_sync(kAll, before);
    before = scan(before);
    if (n > kList) {
      // The lanes say little when there are few of them: close in on a score that leaves a list's worth.
      uint32_t lo = ordered(least), hi = first;  // too many from lo on
      least = most;
      n = __reduce_add_sync(kAll, select());
      while (n <= a.K && hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        least = unordered(mid);
        n = __reduce_add_sync(kAll, select());
        if (n > kList) {
          lo = mid;
          n = 0;
        } else if (n <= a.K) {
          hi = mid;
        }
      }
      before = scan(select());
      if (n <= a.K) n = kList + 1;  // more equal scores than the list holds
      bisected = true;
    }
    if (n <= kList) {
      // by expert index, so that among equal scores the earlier candidate is the lower expert
      store_lane<NV>(sc.scores, lane, c);
      int i = before - __popc(mask);
      while (mask) {
        const int j = __ffs(mask) - 1;
        mask &= mask - 1;
        sc.value[i] = sc.scores[e0 + j];
        sc.expert[i] = e0 + j;
        ++i;
      }
      if (lane < 4 && n + lane < kList) sc.value[n + lane] = -kInf;  // the list in fours
      __syncwarp();
      int rank[2] = {0, 0};
      float (&v)[2] = z;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int me = lane + 32 * h;
        if (32 * h >= n) break;
        v[h] = me < n ? sc.value[me] : kInf;
        for (int q = 0; q < n; q += 4) {
          const float4 u = *reinterpret_cast<const float4*>(sc.value + q);
          rank[h] += u.x > v[h] ? 1 : 0;
          rank[h] += u.y > v[h] ? 1 : 0;
          rank[h] += u.z > v[h] ? 1 : 0;
          rank[h] += u.w > v[h] ? 1 : 0;
        }
      }
      // without equal scores the ranks are 0 .. n - 1 (a lane behind the list has none above its infinity)
      if (static_cast<int>(__reduce_add_sync(kAll, rank[0] + rank[1])) != n * (n - 1) / 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int me = lane + 32 * h;
          for (int q = 0; q < me && me < n; ++q) rank[h] += sc.value[q] == v[h] ? 1 : 0;
        }
        __syncwarp();
      }
      if (biased) {
        // in order of rank: a chosen one within the error bound of the next is decided in FP64
        bool tie = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h < n) sc.scores[rank[h]] = v[h];
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)  // (an infinite score is near to every other)
          if (lane + 32 * h < n && rank[h] < a.K && rank[h] + 1 < n) {
            const float next = sc.scores[rank[h] + 1];
            tie |= !(v[h] - next > near_of(err, v[h], next));
            // (this cut was taken where it fell: what lies below it may have to be looked at too)
            if (bisected && rank[h] == a.K - 1) close = !(v[h] - least > near_of(err, v[h], least));
          }
        close = __any_sync(kAll, close);
        if (!close && __any_sync(kAll, tie)) {
          const int2 ranks = decide_candidates<L, NV>(a, row, lane, scratch, top, n);
          rank[0] = ranks.x;
          rank[1] = ranks.y;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!close && lane + 32 * h < n && rank[h] < a.K) {
          id[h] = sc.expert[lane + 32 * h];
          place[h] = rank[h];
        }
      }
      __syncwarp();  // the list is free for the next token
    }
  }
  if (!close && n > kList) {
    // Many equal scores, or K of the list's length: one expert after the other.
    float last = kInf;
    const int rounds = biased ? a.K + 1 : a.K;  // one more, to see how near the first one left out is
    for (int k = 0; k < rounds && !close; ++k) {
      float best = c[0];
      int at = 0;
#pragma unroll
      for (int j = 1; j < NV; ++j)
        if (c[j] > best) {
          best = c[j];
          at = j;
        }
      const float v = warp_max(best);
      if (!(v > -kInf)) break;
      if (biased) {
        if (k > 0 && !(last - v > near_of(err, last, v))) close = true;
        if (k == a.K) break;
        last = v;
      }
      const int owner = __ffs(__ballot_sync(kAll, best == v)) - 1;
      if (lane == owner) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (j == at) c[j] = -kInf;
      }
      const int chosen = __shfl_sync(kAll, e0 + at, owner);
      if (lane == (k & 31)) (k < 32 ? id[0] : id[1]) = chosen;
    }
    n = kList;  // both places of a lane may be taken
    reload = true;
  }
  if (GENERAL && close) {
    const int2 ids = slow_choice<L, NV>(a, row, lane);
    id[0] = ids.x;
    id[1] = ids.y;
    n = kList;
    reload = true;
  }

  // The weights, from the chosen logits, in FP32.  Halves: experts in a lane's second place are rare.
  const bool two = n > 32;
  float w[2] = {0.0f, 0.0f};
  if (reload && id[0] >= 0) z[0] = clean(static_cast<float>(row[id[0]]));
  if (reload && two && id[1] >= 0) z[1] = clean(static_cast<float>(row[id[1]]));
  if (id[0] < 0) z[0] = -kInf;
  if (id[1] < 0) z[1] = -kInf;
  taken = __popc(__ballot_sync(kAll, id[0] >= 0)) + (two ? __popc(__ballot_sync(kAll, id[1] >= 0)) : 0);
  if (a.renormalize) {
    // softmax: over the chosen logits.  sigmoid: over the logarithms of the chosen scores, so that small scores
    // keep their ratios; directly while FP32 holds them in full.
    float m = 0.0f;
    const bool direct = !softmax && !__any_sync(kAll, (id[0] >= 0 && z[0] < -60.0f) || (id[1] >= 0 && z[1] < -60.0f));
    if (!direct) {
      if (!softmax) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (id[h] >= 0) z[h] = fminf(z[h], 0.0f) - log1pf(expf(-fabsf(z[h])));
      }
      m = warp_max(fmaxf(z[0], z[1]));
    }
    auto weigh = [&](float v) { return direct ? fast_rcp(1.0f + expf(-v)) : v == m ? 1.0f : expf(v - m); };
    if (id[0] >= 0) w[0] = weigh(z[0]);
    if (two && id[1] >= 0) w[1] = weigh(z[1]);
    const float sum = warp_sum(w[0] + w[1]);
    const float over = sum > 0.0f ? a.scale * fast_rcp(sum) : 0.0f;
    w[0] *= over;
    w[1] *= over;
  } else {
    auto weigh = [&](float v) {
      return (softmax ? (v == top ? 1.0f : expf(v - top)) * inv : __fdiv_rn(1.0f, 1.0f + expf(-v))) * a.scale;
    };
    if (id[0] >= 0) w[0] = weigh(z[0]);
    if (two && id[1] >= 0) w[1] = weigh(z[1]);
  }
  const int64_t r = t * a.K;
  if (id[0] >= 0) {
    a.expert_ids[r + place[0]] = id[0];
    store_any(a.expert_scale, r + place[0], a.scale_dtype, w[0]);
  }
  if (two && id[1] >= 0) {
    a.expert_ids[r + place[1]] = id[1];
    store_any(a.expert_scale, r + place[1], a.scale_dtype, w[1]);
  }
  // places that no expert is left for
  for (int k = taken + lane; k < a.K; k += 32) {
    a.expert_ids[r + k] = -1;
    store_any(a.expert_scale, r + k, a.scale_dtype, 0.0f);
  }
}

// ---------------------------------------------------------------------------------------------------
// The expert order
// ---------------------------------------------------------------------------------------------------

// Finishes the order of chunk `b` of `chunks`, which holds `routes` routes from r0 on: `before[e]` routes of expert e lie
// in earlier chunks, `total[e]` in all; route(i, rank) gives route i's expert (-1: none) and its rank within the chunk.
// off: E + 1 ints, warp_sums: 32 ints of shared memory.
template <typename F>
__device__ __forceinline__ void finish_order(const mfr_route_args& a, int b, int chunks, int64_t r0, int64_t routes, const int* before,
                                             const int* total, int* off, int* warp_sums, F route) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  // exclusive sum over the experts of their padded rows: 32 experts a warp, then the warps' sums
  const int parts = (a.E + 31) / 32;  // at most 32
  for (int i = warp; i < parts; i += nwarps) {
    const int e = i * 32 + lane;
    int rows = e < a.E ? total[e] : 0;
    if (a.row_align > 1) rows = static_cast<int>((static_cast<unsigned>(rows) + a.row_align - 1) / a.row_align * a.row_align);
    int sum = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, sum, o);
      if (lane >= o) sum += v;
    }
    if (e < a.E) off[e] = sum - rows;
    if (lane == 31) warp_sums[i] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    const int v = lane < parts ? warp_sums[lane] : 0;
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kAll, sum, o);
      if (lane >= o) sum += u;
    }
    __syncwarp();
    warp_sums[lane] = sum - v;
    if (lane == 31) off[a.E] = sum;
  }
  __syncthreads();
  auto start = [&](int e) { return e < a.E ? off[e] + warp_sums[e >> 5] : off[e]; };
  for (int64_t i = tid; i < routes; i += blockDim.x) {
    int rank = 0;
    const int e = route(i, rank);
    int row = -1;
    if (e >= 0) {
      row = start(e) + before[e] + rank;
      a.row_route[row] = static_cast<int>(r0 + i);
    }
    a.perm_idx[r0 + i] = row;
  }
  if (b == 0) {
    for (int e = tid; e <= a.E; e += blockDim.x) {
      a.expert_offsets[e] = start(e);
      if (e < a.E) a.expert_counts[e] = total[e];
    }
  }
  // rows of no route: the padding behind each expert's routes, and everything behind the last expert
  if (a.row_align > 1)
    for (int e = b * nwarps + warp; e < a.E; e += chunks * nwarps)
      for (int row = start(e) + total[e] + lane; row < start(e + 1); row += 32) a.row_route[row] = -1;
  for (int64_t row = off[a.E] + static_cast<int64_t>(b) * blockDim.x + tid; row < a.num_rows; row += static_cast<int64_t>(chunks) * blockDim.x)
    a.row_route[row] = -1;
}

// The tokens [t0, t1) of chunk b.
__device__ __forceinline__ void chunk_of(const RouteParams& p, int b, int64_t& t0, int64_t& t1) {
  t0 = static_cast<int64_t>(p.chunk) * b + min(b, p.extra);
  t1 = t0 + p.chunk + (b < p.extra ? 1 : 0);
}

// Cluster barrier with release and acquire of shared memory, and a load from a peer's shared memory.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ int load_peer(const int* local, uint32_t rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

template <int NV>
constexpr int kRouteThreads = NV <= 8 ? 1024 : 512;

// Shared memory: each warp's scratch, the biases, and for the order the bitmap, the counts (of the chunk, of the chunks
// before it, of all), the offsets, the scan's warp sums and a segment's experts.
constexpr uint16_t kNoExpert = 0xffff;
struct OrderSmem {
  uint32_t* bits;   // [E][kSegWords]
  int *count, *before, *total, *off, *warp_sums;
  uint16_t* chosen; // [kSegTokens][K]
};
__host__ __device__ inline int order_smem_bytes(int E, int K) {
  return E * kSegWords * 4 + 3 * E * 4 + (E + 1) * 4 + 32 * 4 + kSegTokens * K * 2;
}
__device__ __forceinline__ OrderSmem order_smem(uint8_t* base, int E) {
  OrderSmem o;
  o.bits = reinterpret_cast<uint32_t*>(base);
  o.count = reinterpret_cast<int*>(o.bits + E * kSegWords);
  o.before = o.count + E;
  o.total = o.before + E;
  o.warp_sums = o.total + E;
  o.off = o.warp_sums + 32;
  o.chosen = reinterpret_cast<uint16_t*>(o.off + E + 1);
  return o;
}

template <typename L, int NV, bool GENERAL>
__global__ void __launch_bounds__(kRouteThreads<NV>, 1) route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const mfr_route_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, nwarps = blockDim.x >> 5;
  const int warp = __shfl_sync(kAll, tid >> 5, 0);  // so that the compiler knows it to be the same for the warp
  uint8_t* scratch = smem + warp * kScratchBytes<NV>;
  float* bias = reinterpret_cast<float*>(smem + nwarps * kScratchBytes<NV>);
  const OrderSmem o = order_smem(reinterpret_cast<uint8_t*>(bias + (GENERAL ? 32 * NV : 0)), a.E);
  const bool order = a.expert_offsets != nullptr;
  int64_t t0, t1;
  chunk_of(p, blockIdx.x, t0, t1);
  if (order) {
    for (int i = tid; i < a.E * kSegWords; i += blockDim.x) o.bits[i] = 0;
    for (int i = tid; i < a.E; i += blockDim.x) o.count[i] = 0;
  }
  pdl_launch_dependents();
  pdl_wait();
  if (GENERAL)
    for (int e = tid; e < 32 * NV; e += blockDim.x) bias[e] = a.bias != nullptr && e < a.E ? a.bias[e] : 0.0f;
  if (GENERAL || order) __syncthreads();
  // the rank of route i (token i / K of the segment) of expert e among the segment's routes of that expert
  auto rank_of = [&](int i, int e) {
    const int token = i / a.K;
    const uint32_t* bits = o.bits + e * kSegWords;
    int rank = __popc(bits[token >> 5] & ((1u << (token & 31)) - 1));
    for (int w = 0; w < (token >> 5); ++w) rank += __popc(bits[w]);
    return rank;
  };
  for (int64_t seg = t0; seg < t1; seg += kSegTokens) {
    const int64_t end = seg + kSegTokens < t1 ? seg + kSegTokens : t1;
    for (int64_t t = seg + warp; t < end; t += nwarps) {
      int id[2], place[2], taken;
      float x[NV];
      load_logits<L, NV>(static_cast<const L*>(a.logits) + t * a.logits_stride, lane * NV, a.E, x);
      route_token<L, NV, GENERAL>(p, t, x, lane, bias, scratch, id, place, taken);
      if (order) {
        const int i = static_cast<int>(t - seg);
        uint16_t* mine = o.chosen + i * a.K;
        for (int k = taken + lane; k < a.K; k += 32) mine[k] = kNoExpert;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (id[h] >= 0) {
            mine[place[h]] = static_cast<uint16_t>(id[h]);
            atomicOr(&o.bits[id[h] * kSegWords + (i >> 5)], 1u << (i & 31));
          }
        }
      }
    }
    if (!order) continue;
    __syncthreads();
    if (!p.clustered) {
      const int routes = static_cast<int>(end - seg) * a.K;
      for (int i = tid; i < routes; i += blockDim.x) {
        const int e = o.chosen[i];
        a.perm_idx[seg * a.K + i] = e == kNoExpert ? -1 : o.count[e] + rank_of(i, e);
      }
      __syncthreads();
    }
    for (int e = tid; e < a.E; e += blockDim.x) {
      int n = 0;
#pragma unroll
      for (int w = 0; w < kSegWords; ++w) {
        n += __popc(o.bits[e * kSegWords + w]);
        if (!p.clustered) o.bits[e * kSegWords + w] = 0;
      }
      o.count[e] += n;
    }
    __syncthreads();
  }
  if (!order) return;
  if (!p.clustered) {
    for (int e = tid; e < a.E; e += blockDim.x) static_cast<int*>(a.workspace)[static_cast<int64_t>(blockIdx.x) * a.E + e] = o.count[e];
    return;
  }
  // one cluster holds the whole batch, a segment a CTA
  const int chunks = gridDim.x, b = blockIdx.x;
  if (chunks > 1) cluster_barrier();
  for (int e = tid; e < a.E; e += blockDim.x) {
    int before = 0, total = 0;
    for (int c = 0; c < chunks; ++c) {
      const int v = chunks > 1 ? load_peer(o.count + e, c) : o.count[e];
      total += v;
      if (c < b) before += v;
    }
    o.before[e] = before;
    o.total[e] = total;
  }
  if (chunks > 1) {
    cluster_barrier();  // (no CTA leaves while a peer reads its counts)
  } else {
    __syncthreads();
  }
  finish_order(a, b, chunks, t0 * a.K, (t1 - t0) * a.K, o.before, o.total, o.off, o.warp_sums, [&](int64_t i, int& rank) {
    const int e = o.chosen[i];
    if (e == kNoExpert) return -1;
    rank = rank_of(static_cast<int>(i), e);
    return e;
  });
}

constexpr int kOrderThreads = 1024;
constexpr int kOrderParts = 4096;  // partial counts of an expert, times the experts, at most

// Adds the chunks' counts and finishes the order of chunk blockIdx.x.  Every CTA reads all counts (152 x 256 of them 156
// KB, from L2) rather than wait for another launch to add them once: about 5.5 us, latency from the first load to the
// last store.
__global__ void __launch_bounds__(kOrderThreads, 1) order_kernel(const __grid_constant__ RouteParams p) {
  __shared__ int before[MFR_MAX_EXPERTS], total[MFR_MAX_EXPERTS], off[MFR_MAX_EXPERTS + 1], warp_sums[32];
  __shared__ int4 part_before[kOrderParts / 4], part_total[kOrderParts / 4];
  const mfr_route_args& a = p.a;
  const int tid = threadIdx.x, b = blockIdx.x, chunks = gridDim.x;
  int64_t t0, t1;
  chunk_of(p, b, t0, t1);
  const int64_t r0 = t0 * a.K, routes = (t1 - t0) * a.K;
  // columns of the count matrix, four at a time when its rows allow; the threads split the rows too
  const int wide = a.E % 4 == 0 ? 4 : 1, cols = a.E / wide;
  const int parts = min(kOrderThreads / cols, 32), part = tid / cols, c = tid - part * cols;
  const int* column = static_cast<const int*>(a.workspace) + c * wide;
  pdl_launch_dependents();
  pdl_wait();
  // this thread's first route, on its way while the counts are added
  const int e_first = tid < routes ? a.expert_ids[r0 + tid] : -1, rank_first = tid < routes ? a.perm_idx[r0 + tid] : 0;
  if (part < parts) {
    if (wide == 4) {
      int4 n = make_int4(0, 0, 0, 0), m = n;
#pragma unroll 10
      for (int i = part; i < chunks; i += parts) {
        const int4 v = *reinterpret_cast<const int4*>(column + i * a.E);
        n.x += v.x, n.y += v.y, n.z += v.z, n.w += v.w;
        if (i < b) m.x += v.x, m.y += v.y, m.z += v.z, m.w += v.w;
      }
      part_total[part * cols + c] = n;
      part_before[part * cols + c] = m;
    } else {
      int n = 0, m = 0;
#pragma unroll 10
      for (int i = part; i < chunks; i += parts) {
        const int v = column[i * a.E];
        n += v;
        if (i < b) m += v;
      }
      reinterpret_cast<int*>(part_total)[part * a.E + c] = n;
      reinterpret_cast<int*>(part_before)[part * a.E + c] = m;
    }
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kOrderThreads) {
    int n = 0, m = 0;
    for (int i = 0; i < parts; ++i) {
      n += reinterpret_cast<const int*>(part_total)[i * a.E + e];
      m += reinterpret_cast<const int*>(part_before)[i * a.E + e];
    }
    total[e] = n;
    before[e] = m;
  }
  __syncthreads();
  finish_order(a, b, chunks, r0, routes, before, total, off, warp_sums, [&](int64_t i, int& rank) {
    if (i == tid) {
      rank = rank_first;
      return e_first;
    }
    rank = a.perm_idx[r0 + i];
    return a.expert_ids[r0 + i];
  });
}

template <typename L, int NV, bool GENERAL>
cudaError_t launch_route_nv(const mfr_route_args& a, cudaStream_t stream) {
  const bool order = a.expert_offsets != nullptr, pdl = a.flags & MFR_FLAG_PDL;
  constexpr int kThreads = kRouteThreads<NV>;
  const int fixed = kThreads / 32 * kScratchBytes<NV> + (GENERAL ? 32 * NV * 4 : 0);
  const int smem = fixed + (order ? order_smem_bytes(a.E, a.K) : 0);
  auto kern = route_kernel<L, NV, GENERAL>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = allow_smem<route_kernel<L, NV, GENERAL>>(fixed + order_smem_bytes(NV * 32, MFR_MAX_TOP_K));
  if (e != cudaSuccess) return e;
  const int chunks = route_chunks(a.T, a.E, order);
  RouteParams p{a, a.E / a.num_groups, -1, order && chunks <= kRouteCluster, a.T / chunks, a.T % chunks};
  for (int w = 0; w <= 5; ++w)
    if (p.group_size == NV << w) p.width_log2 = w;
  e = launch_pdl<RouteParams>(kern, dim3(chunks), kThreads, smem, pdl, stream, p, p.clustered ? chunks : 1);
  if (e != cudaSuccess || !order || p.clustered) return e;
  return launch_pdl<RouteParams>(order_kernel, dim3(chunks), kOrderThreads, 0, pdl, stream, p);
}

template <typename L, int NV>
cudaError_t launch_route_g(const mfr_route_args& a, cudaStream_t stream) {
  return a.bias != nullptr || a.num_groups > 1 ? launch_route_nv<L, NV, true>(a, stream) : launch_route_nv<L, NV, false>(a, stream);
}

template <typename L>
cudaError_t launch_route_t(const mfr_route_args& a, cudaStream_t stream) {
  if (a.E <= 32) return launch_route_g<L, 1>(a, stream);
  if (a.E <= 64) return launch_route_g<L, 2>(a, stream);
  if (a.E <= 128) return launch_route_g<L, 4>(a, stream);
  if (a.E <= 256) return launch_route_g<L, 8>(a, stream);
  if (a.E <= 512) return launch_route_g<L, 16>(a, stream);
  return launch_route_g<L, 32>(a, stream);
}

// ---------------------------------------------------------------------------------------------------
// The gradient
// ---------------------------------------------------------------------------------------------------

constexpr int kGradThreads = 256;

// Writes a lane's NV values of a row, in vectors when all of them exist and the address allows.
template <typename L, int NV>
__device__ __forceinline__ void store_logits(L* row, int e0, int E, const float (&v)[NV]) {
  constexpr int kBytes = NV * static_cast<int>(sizeof(L));
  constexpr int kVec = kBytes >= 16 ? 16 : kBytes;
  L* p = row + e0;
  if constexpr (kVec >= 4) {
    if (e0 + NV <= E && (reinterpret_cast<uintptr_t>(p) & (kVec - 1)) == 0) {
      uint32_t raw[kBytes / 4];
#pragma unroll
      for (int i = 0; i < kBytes / 4; ++i) {
        if constexpr (sizeof(L) == 4)
          raw[i] = __float_as_uint(v[i]);
        else
          raw[i] = Act<L>::pack(v[2 * i], v[2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < kBytes / kVec; ++i) {
        if constexpr (kVec == 16)
          reinterpret_cast<uint4*>(p)[i] = make_uint4(raw[4 * i], raw[4 * i + 1], raw[4 * i + 2], raw[4 * i + 3]);
        else if constexpr (kVec == 8)
          reinterpret_cast<uint2*>(p)[i] = make_uint2(raw[2 * i], raw[2 * i + 1]);
        else
          reinterpret_cast<uint32_t*>(p)[i] = raw[i];
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (e0 + j < E) {
      if constexpr (sizeof(L) == 4)
        p[j] = v[j];
      else if constexpr (std::is_same<L, __nv_bfloat16>::value)
        p[j] = __float2bfloat16_rn(v[j]);
      else
        p[j] = __float2half_rn(v[j]);
    }
  }
}

// One warp a token.  The chosen experts' gradients meet their experts' lanes through a row of shared memory, all zeros
// between tokens; the other experts get their share (softmax without renormalisation) or zeros.
//   softmax            dx_e = s_e (ds_e - sum_k ds_k s_k)       ds_k = scale * dw_k, 0 for experts not chosen
//   softmax, renorm    dx_k = p_k (ds_k - sum_j ds_j p_j)       p = softmax over the chosen logits
//   sigmoid            dx_k = ds_k s_k (1 - s_k)
//   sigmoid, renorm    dx_k = p_k (1 - s_k) (ds_k - sum_j ds_j p_j)   p = s / sum s
// Bound by HBM: the logits are read (softmax without renormalisation; else only the chosen ones) and the gradient
// written once.  16384 tokens of 256 experts, FP32 softmax without renormalisation, 35 MB: 8.5 us in a graph (5.1 us at
// the copy bandwidth; about 3 us are the launch and the first loads).  With scalar loads and the row read three times it
// took 15.4 us, without the next token's request 9.4.
template <typename L, int NV>
__global__ void __launch_bounds__(kGradThreads) route_grad_kernel(const __grid_constant__ mfr_route_backward_args a) {
  __shared__ __align__(16) float rows[kGradThreads / 32][32 * NV];
  const int lane = threadIdx.x & 31, nwarps = kGradThreads / 32, e0 = lane * NV;
  const int warp = __shfl_sync(kAll, static_cast<int>(threadIdx.x >> 5), 0);  // known to be the same for the warp
  float* buf = rows[warp];
  const bool softmax = a.score == MFR_SCORE_SOFTMAX, dense = softmax && !a.renormalize, two = a.K > 32;
  if (!dense) {
    for (int e = lane; e < 32 * NV; e += 32) buf[e] = 0.0f;  // zeros between tokens
    __syncwarp();
  }
  pdl_launch_dependents();
  pdl_wait();
  // What a token needs, requested while the one before it is worked on.
  struct Token {
    float v[NV];  // the logits (dense; with many experts a lane they are loaded when they are needed)
    int id[2];
    float d[2];
  };
  constexpr bool kAhead = NV <= 8;
  auto load_row = [&](int64_t t, float (&v)[NV]) {
    load_logits<L, NV>(static_cast<const L*>(a.logits) + t * a.logits_stride, e0, a.E, v);
  };
  auto load = [&](int64_t t, Token& z) {
    if (dense && kAhead) load_row(t, z.v);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = lane + 32 * i;
      const bool in = (i == 0 || two) && k < a.K;
      z.id[i] = in ? a.expert_ids[t * a.K + k] : -1;
      z.d[i] = in ? load_any(a.d_scale, t * a.K + k, a.scale_dtype) : 0.0f;
      if (z.id[i] < 0 || z.id[i] >= a.E) {
        z.id[i] = -1;
        z.d[i] = 0.0f;
      }
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * nwarps + warp;
  const int64_t step = static_cast<int64_t>(gridDim.x) * nwarps;
  if (t >= a.T) return;
  Token z;
  load(t, z);
  for (; t < a.T; t += step) {
    const L* row = static_cast<const L*>(a.logits) + t * a.logits_stride;
    if (dense && !kAhead) load_row(t, z.v);
    Token next;
    if (t + step < a.T) load(t + step, next);
    float (&v)[NV] = z.v;
    const int (&id)[2] = z.id;
    float d[2] = {z.d[0] * a.scale, z.d[1] * a.scale}, g[2] = {0.0f, 0.0f}, inner = 0.0f;
    if (dense) {
      float m = v[0], sum = 0.0f;
#pragma unroll
      for (int j = 1; j < NV; ++j) m = fmaxf(m, v[j]);
      const float top = warp_max(m);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        v[j] = !(v[j] > -kInf) ? 0.0f : v[j] == top ? 1.0f : fast_exp2((v[j] - top) * kLog2e);
        sum += v[j];
      }
      store_lane<NV>(buf, lane, v);
      sum = warp_sum(sum);
      const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float p = id[i] >= 0 ? buf[id[i]] * inv : 0.0f;
        g[i] = p * d[i];
      }
      inner = warp_sum(g[0] + g[1]) * inv;
      // the share that every expert has
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] *= -inner;
      __syncwarp();
      store_lane<NV>(buf, lane, v);
      __syncwarp();
    } else {
      float x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) x[i] = id[i] >= 0 ? clean(static_cast<float>(row[id[i]])) : -kInf;
      // The weights p over the chosen experts (sigmoid without renormalisation: s), and 1 - s of the sigmoid.  Softmax from
      // the logits, sigmoid from the logarithms of the scores.
      float p[2] = {0.0f, 0.0f}, q[2] = {1.0f, 1.0f};
      if (!softmax) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if ((i == 0 || two) && id[i] >= 0) {
            q[i] = __fdiv_rn(1.0f, 1.0f + expf(x[i]));
            if (a.renormalize)
              x[i] = fminf(x[i], 0.0f) - log1pf(expf(-fabsf(x[i])));
            else
              p[i] = __fdiv_rn(1.0f, 1.0f + expf(-x[i]));
          }
        }
      }
      if (a.renormalize) {
        const float m = warp_max(fmaxf(x[0], x[1]));
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if ((i == 0 || two) && x[i] > -kInf) p[i] = x[i] == m ? 1.0f : expf(x[i] - m);
        const float sum = warp_sum(p[0] + p[1]);
        const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        p[0] *= inv;
        p[1] *= inv;
        inner = warp_sum(d[0] * p[0] + d[1] * p[1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) g[i] = p[i] * q[i] * (d[i] - inner);
    }
    // Distinct experts at once; an expert named twice gets its gradients place by place.
    const unsigned same = __match_any_sync(kAll, id[0]);  // (every lane takes part)
    const bool twice = id[0] >= 0 && (same & (kAll >> (31 - lane))) != 1u << lane;
    if (two || __any_sync(kAll, twice)) {
      for (int k = 0; k < a.K; ++k) {
        if (lane == (k & 31)) {
          const int e = k < 32 ? id[0] : id[1];
          if (e >= 0) buf[e] += k < 32 ? g[0] : g[1];
        }
        __syncwarp();
      }
    } else if (id[0] >= 0) {
      buf[id[0]] += g[0];
    }
    __syncwarp();
    load_lane<NV>(buf, lane, v);
    __syncwarp();
    if (!dense) {
      if (id[0] >= 0) buf[id[0]] = 0.0f;
      if (id[1] >= 0) buf[id[1]] = 0.0f;
      __syncwarp();
    }
    store_logits<L, NV>(static_cast<L*>(a.d_logits) + t * a.d_logits_stride, e0, a.E, v);
    z = next;
  }
}

template <typename L, int NV>
cudaError_t launch_route_backward_nv(const mfr_route_backward_args& a, cudaStream_t stream) {
  const int per = kGradThreads / 32;
  const int64_t want = (static_cast<int64_t>(a.T) + per - 1) / per;
  // (so few CTAs that a warp has a next token to request: 8.5 us at 5 an SM, 8.6 at 8 or 16, 10.6 at 4, for the batch above)
  const int blocks = static_cast<int>(want < 152 * 5 ? want : 152 * 5);
  return launch_pdl<mfr_route_backward_args>(route_grad_kernel<L, NV>, dim3(blocks), kGradThreads, 0, a.flags & MFR_FLAG_PDL, stream, a);
}

template <typename L>
cudaError_t launch_route_backward_t(const mfr_route_backward_args& a, cudaStream_t stream) {
  if (a.E <= 32) return launch_route_backward_nv<L, 1>(a, stream);
  if (a.E <= 64) return launch_route_backward_nv<L, 2>(a, stream);
  if (a.E <= 128) return launch_route_backward_nv<L, 4>(a, stream);
  if (a.E <= 256) return launch_route_backward_nv<L, 8>(a, stream);
  if (a.E <= 512) return launch_route_backward_nv<L, 16>(a, stream);
  return launch_route_backward_nv<L, 32>(a, stream);
}

}  // namespace

cudaError_t launch_route(const mfr_route_args& a, cudaStream_t stream) {
  switch (a.logits_dtype) {
    case MFR_BF16: return launch_route_t<__nv_bfloat16>(a, stream);
    case MFR_FP16: return launch_route_t<__half>(a, stream);
    default: return launch_route_t<float>(a, stream);
  }
}

cudaError_t launch_route_backward(const mfr_route_backward_args& a, cudaStream_t stream) {
  switch (a.logits_dtype) {
    case MFR_BF16: return launch_route_backward_t<__nv_bfloat16>(a, stream);
    case MFR_FP16: return launch_route_backward_t<__half>(a, stream);
    default: return launch_route_backward_t<float>(a, stream);
  }
}

}  // namespace mfr
