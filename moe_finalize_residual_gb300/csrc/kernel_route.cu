// Routing to experts: scores, expert groups, the K best experts of each token, their weights, and the
// expert order of the routes; and the gradient of the weights to the logits.
//
// One warp takes one token.  Lane l holds the NV consecutive experts from l * NV on, so among equal scores
// the lowest lane, and within it the lowest slot, is the lowest expert index.
//
// The order of the chosen experts is that of 64-bit choice scores.  Without a bias a score orders as its
// logit, and the logits are compared as they are.  With a bias (and for group scores that are sums) the
// scores are computed in FP32 with a proven bound on their error; where two neighbours in the order lie
// closer than the bound, the token is decided again in FP64 (slow_choice), which random inputs need about
// once in a thousand tokens.
//
// The expert order is a stable counting sort.  A CTA takes a contiguous chunk of tokens and marks each
// route in a bitmap [expert][token of the segment]: a route's rank among its expert's routes is the number
// of marks below its own, so the marks may be set in any order (atomicOr) with the same result.  The chunks'
// counts meet in a second kernel (order_kernel), which adds those of the chunks before its own; a batch of
// one chunk does both in one launch.
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

// The two best of two pairs of best values.
template <typename F>
__device__ __forceinline__ void merge_top2(F& a, F& b, F a2, F b2) {
  const F lo = a < a2 ? a : a2;
  const F hi = b > b2 ? b : b2;
  a = a > a2 ? a : a2;
  b = lo > hi ? lo : hi;
}

// The group score of a group's two best choice scores (-inf: none).
template <typename F>
__device__ __forceinline__ F group_score(F best, F second, bool top2) {
  return top2 && second > static_cast<F>(-kInf) ? best + second : best;
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
// ids of places l and l + 32.
template <typename L, int NV>
__device__ __noinline__ void slow_choice(const mfr_route_args& a, const L* row, int lane, int& id0, int& id1) {
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
  id0 = id1 = -1;
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

// The groups whose scores lie within `tol` of the border between kept and dropped ones, decided again in FP64.
// sc.scores holds the values that the groups compare, lane g group g's score and second best value; `in`: whether
// it is kept.  Returns the groups kept, or 0 when too many values matter.
template <typename L>
__device__ __noinline__ unsigned decide_groups(const RouteParams& p, const L* row, int lane, const Scratch& sc, float top, float mine,
                                               float second, bool in, float worst, float best_out, float tol) {
  const mfr_route_args& a = p.a;
  const bool top2 = a.group_score == MFR_GROUP_TOP2, biased = a.bias != nullptr;
  const bool here = lane < a.num_groups && mine > -kInf;
  const unsigned kept = __ballot_sync(kAll, in);
  const unsigned band = __ballot_sync(kAll, here && !(in ? mine - best_out > tol : worst - mine > tol));
  // the values that may be among a group's two best
  int n = 0, begin = 0, end = 0;
  for (unsigned m = band; m; m &= m - 1) {
    const int g = __ffs(m) - 1;
    const float least = fmaxf(__shfl_sync(kAll, top2 ? second : mine, g) - tol, -3.402823466e38f);
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
template <typename L>
__device__ __noinline__ void decide_candidates(const mfr_route_args& a, const L* row, int lane, const Scratch& sc, float top, int n,
                                               int& rank0, int& rank1) {
  const double inv = 1.0 / score_sum64(a, row, lane, top);
  for (int q = lane; q < n; q += 32) {
    const int e = sc.expert[q];
    sc.wide[q] = ordered64(raw_score64(a.score, clean(static_cast<float>(row[e])), top) * inv + static_cast<double>(a.bias[e]));
  }
  __syncwarp();
  const int64_t v0 = lane < n ? sc.wide[lane] : 0, v1 = lane + 32 < n ? sc.wide[lane + 32] : 0;
  rank0 = rank1 = 0;
  for (int q = 0; q < n; ++q) {
    const int64_t u = sc.wide[q];
    rank0 += (u > v0 || (u == v0 && q < lane)) ? 1 : 0;
    rank1 += (u > v1 || (u == v1 && q < lane + 32)) ? 1 : 0;
  }
}

// Chooses and weighs the experts of one token whose logits are x.  Each lane gets up to two of them: the
// expert id[i] at place[i] of the token's list, or id -1.  `bias`: the experts' biases in shared memory.
template <typename L, int NV>
__device__ __forceinline__ void route_token(const RouteParams& p, int64_t t, float (&x)[NV], int lane, const float* bias,
                                            const Scratch& sc, int (&id)[2], int (&place)[2]) {
  const mfr_route_args& a = p.a;
  const L* row = static_cast<const L*>(a.logits) + t * a.logits_stride;
  const int e0 = lane * NV;
  const bool softmax = a.score == MFR_SCORE_SOFTMAX;
  const bool top2 = a.num_groups > 1 && a.group_score == MFR_GROUP_TOP2;
  const bool biased = a.bias != nullptr;
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
#pragma unroll
    for (int j = 0; j < NV; ++j) c[j] = x[j] > -kInf ? clean(s[j] + bias[e0 + j]) : -kInf;
  }

  bool close = false;  // a decision lies within the error bound and too many experts with it: all in FP64
  if (a.num_groups > 1) {
    const bool sums = top2 && !biased;  // groups compare sums of scores, experts compare logits
    float mine = -kInf, second = -kInf; // lane g: group g's score, and its second best value
    if (p.width_log2 >= 0) {
      float b1 = -kInf, b2 = -kInf;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float v = sums ? (c[j] > -kInf ? s[j] : -kInf) : c[j];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
      for (int o = (1 << p.width_log2) >> 1; o > 0; o >>= 1) {
        const float v1 = __shfl_xor_sync(kAll, b1, o), v2 = __shfl_xor_sync(kAll, b2, o);
        b2 = fmaxf(fminf(b1, v1), fmaxf(b2, v2));
        b1 = fmaxf(b1, v1);
      }
      const int from = (lane << p.width_log2) & 31;
      mine = __shfl_sync(kAll, group_score(b1, b2, top2), from);
      second = __shfl_sync(kAll, b2, from);
      if (lane >= a.num_groups) mine = -kInf;
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) sc.scores[e0 + j] = sums ? (c[j] > -kInf ? s[j] : -kInf) : c[j];
      __syncwarp();
      if (lane < a.num_groups) {
        float b1 = -kInf;
        for (int i = 0; i < p.group_size; ++i) {
          const float v = sc.scores[lane * p.group_size + i];
          second = fmaxf(second, fminf(b1, v));
          b1 = fmaxf(b1, v);
        }
        mine = group_score(b1, second, top2);
      }
      __syncwarp();
    }
    int rank = 0;
#pragma unroll 4
    for (int g = 0; g < a.num_groups; ++g) {
      const float v = __shfl_sync(kAll, mine, g);
      rank += (v > mine || (v == mine && g < lane)) ? 1 : 0;
    }
    const bool in = rank < a.topk_groups && mine > -kInf;
    unsigned kept = __ballot_sync(kAll, in);
    if (top2 || biased) {
      // the kept group nearest to a dropped one
      const float worst = -warp_max(in ? -mine : -kInf);
      const float best_out = warp_max(in ? -kInf : mine);
      const float tol = (top2 ? 4.0f : 2.0f) * err + 2.4e-7f * (fabsf(worst) + fabsf(best_out));
      if (best_out > -kInf && !(worst - best_out > tol)) {
        if (p.width_log2 >= 0) {
#pragma unroll
          for (int j = 0; j < NV; ++j) sc.scores[e0 + j] = sums ? (c[j] > -kInf ? s[j] : -kInf) : c[j];
          __syncwarp();
        }
        kept = decide_groups(p, row, lane, sc, top, mine, second, in, worst, best_out, tol);
        close = kept == 0;
      }
    }
    if (p.width_log2 >= 0) {
      if (!((kept >> (lane >> p.width_log2)) & 1)) {
#pragma unroll
        for (int j = 0; j < NV; ++j) c[j] = -kInf;
      }
    } else {
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
  int n = kList + 1;  // candidates
  if (!close && a.K < 32) {
    // The K + 1 best of the lanes' best bound the K + 1 best experts from below: every expert from there on is a
    // candidate (about 10 of 256 for K = 8), and the candidates are ranked by counting.
    float best = c[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) best = fmaxf(best, c[j]);
    uint32_t key = ordered(best);
    const uint32_t first = __reduce_max_sync(kAll, key);
    uint32_t tau = first;
#pragma unroll 4
    for (int k = 0; k < a.K; ++k) {
      if (key == tau) key = 0;
      tau = __reduce_max_sync(kAll, key);
    }
    const float most = unordered(first);
    // fewer lanes than that have any: all experts that can be taken are candidates
    const float least = tau > ordered(-kInf) ? unordered(tau) : -3.402823466e38f;
    unsigned mask = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) mask |= c[j] >= least ? 1u << j : 0u;
    int before = __popc(mask);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, before, o);
      if (lane >= o) before += v;
    }
    n = __shfl_sync(kAll, before, 31);
    if (n <= kList) {
      // by expert index, so that among equal scores the earlier candidate is the lower expert
#pragma unroll
      for (int j = 0; j < NV; ++j) sc.scores[e0 + j] = c[j];
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
      float v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int me = lane + 32 * h;
        if (32 * h >= n) break;
        v[h] = me < n ? sc.value[me] : -kInf;
        for (int q = 0; q < n; q += 4) {
          const float4 u = *reinterpret_cast<const float4*>(sc.value + q);
          rank[h] += (u.x > v[h] || (u.x == v[h] && q < me)) ? 1 : 0;
          rank[h] += (u.y > v[h] || (u.y == v[h] && q + 1 < me)) ? 1 : 0;
          rank[h] += (u.z > v[h] || (u.z == v[h] && q + 2 < me)) ? 1 : 0;
          rank[h] += (u.w > v[h] || (u.w == v[h] && q + 3 < me)) ? 1 : 0;
        }
      }
      if (biased) {
        // in order of rank: a chosen one within the error bound of the next is decided in FP64
        const float near = 2.0f * err + 2.4e-7f * fmaxf(fabsf(most), fabsf(least));
        bool tie = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h < n) sc.scores[rank[h]] = v[h];
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)  // (an infinite score is near to every other)
          if (lane + 32 * h < n && rank[h] < a.K && rank[h] + 1 < n) tie |= !(v[h] - sc.scores[rank[h] + 1] > near);
        if (__any_sync(kAll, tie)) decide_candidates(a, row, lane, sc, top, n, rank[0], rank[1]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (lane + 32 * h < n && rank[h] < a.K) {
          id[h] = sc.expert[lane + 32 * h];
          place[h] = rank[h];
        }
      }
      __syncwarp();  // the list is free for the next token
    }
  }
  if (!close && n > kList) {
    // Many equal scores, or K of 32 and more: one expert after the other.
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
        if (k > 0 && !(last - v > 2.0f * err + 1.2e-7f * (fabsf(last) + fabsf(v)))) close = true;
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
  }
  if (close) {
    slow_choice<L, NV>(a, row, lane, id[0], id[1]);
    n = kList;
  }

  // The weights, from the chosen logits, in FP32.  Halves: experts in a lane's second place are rare.
  const bool two = n > 32;
  float w[2] = {0.0f, 0.0f}, z[2] = {-kInf, -kInf};
  if (id[0] >= 0) z[0] = clean(static_cast<float>(row[id[0]]));
  if (two && id[1] >= 0) z[1] = clean(static_cast<float>(row[id[1]]));
  const int taken = __popc(__ballot_sync(kAll, id[0] >= 0)) + (two ? __popc(__ballot_sync(kAll, id[1] >= 0)) : 0);
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
    const float over = sum > 0.0f ? __fdiv_rn(a.scale, sum) : 0.0f;
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

// Finishes the order of one chunk: `before[e]` routes of expert e lie in earlier chunks, `total[e]` in all;
// perm_idx holds each route's rank within the chunk.  off: E + 1 ints of shared memory.
__device__ __forceinline__ void finish_order(const mfr_route_args& a, int64_t r0, int64_t r1, const int* before,
                                             const int* total, int* off, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  // exclusive sum over the experts of their padded rows: 32 experts a warp, then the warps' sums
  const int chunks = (a.E + 31) / 32;  // at most 32
  for (int i = warp; i < chunks; i += nwarps) {
    const int e = i * 32 + lane;
    const int rows = e < a.E ? static_cast<int>((static_cast<int64_t>(total[e]) + a.row_align - 1) / a.row_align * a.row_align) : 0;
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
    const int v = lane < chunks ? warp_sums[lane] : 0;
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kAll, sum, o);
      if (lane >= o) sum += u;
    }
    warp_sums[lane] = sum - v;
    if (lane == 31) off[a.E] = sum;
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += blockDim.x) off[e] += warp_sums[e >> 5];
  __syncthreads();
  for (int64_t r = r0 + tid; r < r1; r += blockDim.x) {
    const int e = a.expert_ids[r];
    int row = -1;
    if (e >= 0) {
      row = off[e] + before[e] + a.perm_idx[r];
      a.row_route[row] = static_cast<int>(r);
    }
    a.perm_idx[r] = row;
  }
  if (blockIdx.x == 0) {
    for (int e = tid; e < a.E; e += blockDim.x) {
      a.expert_offsets[e] = off[e];
      a.expert_counts[e] = total[e];
    }
    if (tid == 0) a.expert_offsets[a.E] = off[a.E];
  }
  // rows of no route: the padding behind each expert's routes, and everything behind the last expert
  if (a.row_align > 1)
    for (int e = blockIdx.x * nwarps + warp; e < a.E; e += gridDim.x * nwarps)
      for (int row = off[e] + total[e] + lane; row < off[e + 1]; row += 32) a.row_route[row] = -1;
  for (int64_t row = off[a.E] + static_cast<int64_t>(blockIdx.x) * blockDim.x + tid; row < a.num_rows;
       row += static_cast<int64_t>(gridDim.x) * blockDim.x)
    a.row_route[row] = -1;
}

// The chunk of tokens of one CTA.
__device__ __forceinline__ void chunk_of(int T, int64_t& t0, int64_t& t1) {
  t0 = static_cast<int64_t>(T) * blockIdx.x / gridDim.x;
  t1 = static_cast<int64_t>(T) * (blockIdx.x + 1) / gridDim.x;
}

template <int NV>
constexpr int route_threads() { return NV <= 8 ? 1024 : 512; }

// Shared memory: each warp's scratch, the biases, and for the order the bitmap, the running counts, the offsets and the
// scan's warp sums.
template <int NV>
int route_smem(int E, bool order) {
  const int scratch = route_threads<NV>() / 32 * kScratchBytes<NV> + 32 * NV * 4;
  return order ? scratch + E * kSegWords * 4 + E * 4 + (E + 1) * 4 + 32 * 4 : scratch;
}

template <typename L, int NV>
__global__ void __launch_bounds__(route_threads<NV>(), 1) route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const mfr_route_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  const Scratch scratch = scratch_of<NV>(smem + warp * kScratchBytes<NV>);
  float* bias = reinterpret_cast<float*>(smem + nwarps * kScratchBytes<NV>);
  uint32_t* bits = reinterpret_cast<uint32_t*>(bias + 32 * NV);
  int* count = reinterpret_cast<int*>(bits + a.E * kSegWords);
  int* off = count + a.E;
  int* warp_sums = off + a.E + 1;
  const bool order = a.expert_offsets != nullptr;
  int64_t t0, t1;
  chunk_of(a.T, t0, t1);
  if (order) {
    for (int i = tid; i < a.E * kSegWords; i += blockDim.x) bits[i] = 0;
    for (int i = tid; i < a.E; i += blockDim.x) count[i] = 0;
  }
  pdl_launch_dependents();
  pdl_wait();
  for (int e = tid; e < 32 * NV; e += blockDim.x) bias[e] = a.bias != nullptr && e < a.E ? a.bias[e] : 0.0f;
  __syncthreads();
  for (int64_t seg = t0; seg < t1; seg += kSegTokens) {
    const int64_t end = seg + kSegTokens < t1 ? seg + kSegTokens : t1;
    for (int64_t t = seg + warp; t < end; t += nwarps) {
      int id[2], place[2];
      float x[NV];
      load_logits<L, NV>(static_cast<const L*>(a.logits) + t * a.logits_stride, lane * NV, a.E, x);
      route_token<L, NV>(p, t, x, lane, bias, scratch, id, place);
      if (order) {
        const int i = static_cast<int>(t - seg);
        if (id[0] >= 0) atomicOr(&bits[id[0] * kSegWords + (i >> 5)], 1u << (i & 31));
        if (id[1] >= 0) atomicOr(&bits[id[1] * kSegWords + (i >> 5)], 1u << (i & 31));
      }
    }
    if (!order) continue;
    __syncthreads();
    const int routes = static_cast<int>(end - seg) * a.K;
    for (int r = tid; r < routes; r += blockDim.x) {
      const int e = a.expert_ids[seg * a.K + r];
      int rank = -1;
      if (e >= 0) {
        const int i = r / a.K;
        rank = count[e] + __popc(bits[e * kSegWords + (i >> 5)] & ((1u << (i & 31)) - 1));
        for (int w = 0; w < (i >> 5); ++w) rank += __popc(bits[e * kSegWords + w]);
      }
      a.perm_idx[seg * a.K + r] = rank;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += blockDim.x) {
      int n = 0;
#pragma unroll
      for (int w = 0; w < kSegWords; ++w) {
        n += __popc(bits[e * kSegWords + w]);
        bits[e * kSegWords + w] = 0;
      }
      count[e] += n;
    }
    __syncthreads();
  }
  if (!order) return;
  if (gridDim.x > 1) {
    for (int e = tid; e < a.E; e += blockDim.x) static_cast<int*>(a.workspace)[blockIdx.x * a.E + e] = count[e];
  } else {
    // one chunk: nothing lies before it (the bitmap is all zeros again and serves as `before`)
    finish_order(a, t0 * a.K, t1 * a.K, reinterpret_cast<const int*>(bits), count, off, warp_sums);
  }
}

constexpr int kOrderThreads = 1024;

// Adds the chunks' counts and finishes the order of chunk blockIdx.x.
__global__ void __launch_bounds__(kOrderThreads, 1) order_kernel(const __grid_constant__ RouteParams p) {
  const mfr_route_args& a = p.a;
  __shared__ int before[MFR_MAX_EXPERTS], total[MFR_MAX_EXPERTS], off[MFR_MAX_EXPERTS + 1], warp_sums[32];
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) before[e] = total[e] = 0;
  __syncthreads();
  pdl_wait();
  // columns of the count matrix: the threads split its rows too, and meet by integer adds (any order)
  const int* ws = static_cast<const int*>(a.workspace);
  const int parts = kOrderThreads / a.E;  // E <= 1024
  const int part = threadIdx.x / a.E, e = threadIdx.x % a.E;
  if (part < parts) {
    int b = 0, n = 0;
#pragma unroll 8
    for (int i = part; i < static_cast<int>(gridDim.x); i += parts) {
      const int v = ws[i * a.E + e];
      n += v;
      if (i < static_cast<int>(blockIdx.x)) b += v;
    }
    atomicAdd(&before[e], b);
    atomicAdd(&total[e], n);
  }
  __syncthreads();
  int64_t t0, t1;
  chunk_of(a.T, t0, t1);
  finish_order(a, t0 * a.K, t1 * a.K, before, total, off, warp_sums);
}

template <typename L, int NV>
cudaError_t launch_route_nv(const mfr_route_args& a, cudaStream_t stream) {
  const bool order = a.expert_offsets != nullptr, pdl = a.flags & MFR_FLAG_PDL;
  const int smem = route_smem<NV>(a.E, order);
  auto kern = route_kernel<L, NV>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, route_smem<NV>(NV * 32, true));
  if (e != cudaSuccess) return e;
  const int blocks = route_blocks(a.T);
  RouteParams p{a, a.E / a.num_groups, -1};
  for (int w = 0; w <= 5; ++w)
    if (p.group_size == NV << w) p.width_log2 = w;
  e = launch_pdl<RouteParams>(kern, dim3(blocks), route_threads<NV>(), smem, pdl, stream, p);
  if (e != cudaSuccess || !order || blocks == 1) return e;
  return launch_pdl<RouteParams>(order_kernel, dim3(blocks), kOrderThreads, 0, pdl, stream, p);
}

template <typename L>
cudaError_t launch_route_t(const mfr_route_args& a, cudaStream_t stream) {
  if (a.E <= 32) return launch_route_nv<L, 1>(a, stream);
  if (a.E <= 64) return launch_route_nv<L, 2>(a, stream);
  if (a.E <= 128) return launch_route_nv<L, 4>(a, stream);
  if (a.E <= 256) return launch_route_nv<L, 8>(a, stream);
  if (a.E <= 512) return launch_route_nv<L, 16>(a, stream);
  return launch_route_nv<L, 32>(a, stream);
}

// ---------------------------------------------------------------------------------------------------
// The gradient
// ---------------------------------------------------------------------------------------------------

constexpr int kGradThreads = 256;

// One warp a token: the chosen experts' gradients go into the warp's row of shared memory, which is then
// written out whole, with the other experts' share (softmax without renormalisation) or zeros.
//   softmax            dx_e = s_e (ds_e - sum_k ds_k s_k)       ds_k = scale * dw_k, 0 for experts not chosen
//   softmax, renorm    dx_k = p_k (ds_k - sum_j ds_j p_j)       p = softmax over the chosen logits
//   sigmoid            dx_k = ds_k s_k (1 - s_k)
//   sigmoid, renorm    dx_k = p_k (1 - s_k) (ds_k - sum_j ds_j p_j)   p = s / sum s
template <typename L>
__global__ void __launch_bounds__(kGradThreads) route_grad_kernel(const __grid_constant__ mfr_route_backward_args a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = kGradThreads / 32;
  float* buf = reinterpret_cast<float*>(smem) + warp * a.E;
  for (int e = lane; e < a.E; e += 32) buf[e] = 0.0f;
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();
  const bool softmax = a.score == MFR_SCORE_SOFTMAX, dense = softmax && !a.renormalize;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * nwarps + warp; t < a.T; t += static_cast<int64_t>(gridDim.x) * nwarps) {
    const L* row = static_cast<const L*>(a.logits) + t * a.logits_stride;
    L* out = static_cast<L*>(a.d_logits) + t * a.d_logits_stride;
    int id[2];
    float x[2], d[2], g[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = lane + 32 * i;
      id[i] = k < a.K ? a.expert_ids[t * a.K + k] : -1;
      if (id[i] >= a.E) id[i] = -1;
      x[i] = id[i] >= 0 ? clean(static_cast<float>(row[id[i]])) : -kInf;
      d[i] = id[i] >= 0 ? load_any(a.d_scale, t * a.K + k, a.scale_dtype) * a.scale : 0.0f;
    }
    float top = -kInf, inv = 0.0f, inner = 0.0f;
    if (dense) {
      for (int e = lane; e < a.E; e += 32) top = fmaxf(top, clean(static_cast<float>(row[e])));
      top = warp_max(top);
      float sum = 0.0f;
      for (int e = lane; e < a.E; e += 32) {
        const float v = clean(static_cast<float>(row[e]));
        if (v > -kInf) sum += v == top ? 1.0f : expf(v - top);
      }
      sum = warp_sum(sum);
      inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    }
    if (softmax) {
      if (!dense) top = warp_max(fmaxf(x[0], x[1]));
      float p[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) p[i] = !(x[i] > -kInf) ? 0.0f : x[i] == top ? 1.0f : expf(x[i] - top);
      if (!dense) {
        const float sum = warp_sum(p[0] + p[1]);
        inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) p[i] *= inv;
      inner = warp_sum(d[0] * p[0] + d[1] * p[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) g[i] = dense ? p[i] * d[i] : p[i] * (d[i] - inner);
    } else {
      float q[2], l[2];  // 1 - s, and the weight p (or s)
#pragma unroll
      for (int i = 0; i < 2; ++i) q[i] = __fdiv_rn(1.0f, 1.0f + expf(x[i]));
      if (a.renormalize) {
#pragma unroll
        for (int i = 0; i < 2; ++i) l[i] = x[i] > -kInf ? fminf(x[i], 0.0f) - log1pf(expf(-fabsf(x[i]))) : -kInf;
        const float m = warp_max(fmaxf(l[0], l[1]) + 0.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i) l[i] = !(l[i] > -kInf) ? 0.0f : l[i] == m ? 1.0f : expf(l[i] - m);
        const float sum = warp_sum(l[0] + l[1]);
        inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        l[0] *= inv;
        l[1] *= inv;
        inner = warp_sum(d[0] * l[0] + d[1] * l[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) l[i] = __fdiv_rn(1.0f, 1.0f + expf(-x[i]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) g[i] = l[i] * q[i] * (d[i] - inner);
    }
    // place by place, so that an expert named twice gets both, in order
    for (int k = 0; k < a.K; ++k) {
      if (lane == (k & 31)) {
        const int i = k >> 5;
        const int e = i ? id[1] : id[0];
        if (e >= 0) buf[e] += i ? g[1] : g[0];
      }
      __syncwarp();
    }
    for (int e = lane; e < a.E; e += 32) {
      float v = buf[e];
      if (dense) {
        const float z = clean(static_cast<float>(row[e]));
        if (z > -kInf) v -= (z == top ? 1.0f : expf(z - top)) * inv * inner;
      }
      buf[e] = 0.0f;
      if constexpr (sizeof(L) == 4)
        out[e] = v;
      else if constexpr (std::is_same<L, __nv_bfloat16>::value)
        out[e] = __float2bfloat16_rn(v);
      else
        out[e] = __float2half_rn(v);
    }
    __syncwarp();
  }
}

template <typename L>
cudaError_t launch_route_backward_t(const mfr_route_backward_args& a, cudaStream_t stream) {
  const int per = kGradThreads / 32;
  const int64_t want = (static_cast<int64_t>(a.T) + per - 1) / per;
  const int blocks = static_cast<int>(want < 152 * 8 ? want : 152 * 8);
  return launch_pdl<mfr_route_backward_args>(route_grad_kernel<L>, dim3(blocks), kGradThreads, per * a.E * 4, a.flags & MFR_FLAG_PDL, stream, a);
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
