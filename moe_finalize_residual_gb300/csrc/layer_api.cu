// C ABI of the operators around the finalize (moe_layer.h): argument validation (nothing is enqueued on
// error), size queries and dispatch to the kernels.
#include <algorithm>
#include <climits>
#include <cstdlib>

#include "layer_launch.h"
#include "mfr_launch.h"

namespace mfr {
namespace {

constexpr int kMaxHeads = 65536;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool any_dtype(int d) { return d == MFR_BF16 || d == MFR_FP16 || d == MFR_FP32; }
uintptr_t dtype_bytes(int d) { return d == MFR_FP32 ? 4 : 2; }

int enqueue_status(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(MFR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return MFR_OK;
}

int check_routes(int T, int K) {
  if (T < 0) return fail(MFR_ERR_INVALID_ARG, "T = %d < 0", T);
  if (K < 1 || K > MFR_MAX_TOP_K) return fail(MFR_ERR_INVALID_ARG, "K = %d outside [1, %d]", K, MFR_MAX_TOP_K);
  if (static_cast<int64_t>(T) * K > INT32_MAX) return fail(MFR_ERR_INVALID_ARG, "T * K = %d * %d is 2^31 or more", T, K);
  return MFR_OK;
}

int check_experts(int E, int K) {
  if (E < 1 || E > MFR_MAX_EXPERTS) return fail(MFR_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, MFR_MAX_EXPERTS);
  if (K > E) return fail(MFR_ERR_INVALID_ARG, "K = %d experts per token of E = %d", K, E);
  return MFR_OK;
}

int check_scoring(int logits_dtype, int scale_dtype, int score, int renormalize) {
  if (!any_dtype(logits_dtype)) return fail(MFR_ERR_UNSUPPORTED, "logits_dtype %d unknown", logits_dtype);
  if (!any_dtype(scale_dtype)) return fail(MFR_ERR_UNSUPPORTED, "scale_dtype %d unknown", scale_dtype);
  if (score != MFR_SCORE_SOFTMAX && score != MFR_SCORE_SIGMOID) return fail(MFR_ERR_UNSUPPORTED, "score %d unknown", score);
  if (renormalize != 0 && renormalize != 1) return fail(MFR_ERR_INVALID_ARG, "renormalize = %d is not 0 or 1", renormalize);
  return MFR_OK;
}

// Element offsets of a strided tensor stay in 64 bits, and T rows of it far below their end.
int check_stride(const char* name, int64_t stride, int E) {
  if (stride < E || stride > (int64_t{1} << 31)) return fail(MFR_ERR_INVALID_ARG, "%s = %lld outside [E = %d, 2^31]", name, static_cast<long long>(stride), E);
  return MFR_OK;
}

int check_flags(uint32_t flags, uint32_t known) {
  if (flags & ~known) return fail(MFR_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags & ~known);
  return MFR_OK;
}

int check_route(const mfr_route_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_routes(a->T, a->K)) != MFR_OK || (st = check_experts(a->E, a->K)) != MFR_OK ||
      (st = check_scoring(a->logits_dtype, a->scale_dtype, a->score, a->renormalize)) != MFR_OK ||
      (st = check_flags(a->flags, MFR_FLAG_PDL)) != MFR_OK || (st = check_stride("logits_stride", a->logits_stride, a->E)) != MFR_OK)
    return st;
  if (a->num_groups < 1 || a->num_groups > MFR_MAX_GROUPS || a->E % a->num_groups != 0)
    return fail(MFR_ERR_INVALID_ARG, "num_groups = %d must divide E = %d and be at most %d", a->num_groups, a->E, MFR_MAX_GROUPS);
  if (a->topk_groups < 1 || a->topk_groups > a->num_groups)
    return fail(MFR_ERR_INVALID_ARG, "topk_groups = %d outside [1, num_groups = %d]", a->topk_groups, a->num_groups);
  if (a->group_score != MFR_GROUP_MAX && a->group_score != MFR_GROUP_TOP2)
    return fail(MFR_ERR_UNSUPPORTED, "group_score %d unknown", a->group_score);
  if (a->row_align < 1) return fail(MFR_ERR_INVALID_ARG, "row_align = %d < 1", a->row_align);
  if (a->expert_offsets != nullptr) {
    if (a->expert_counts == nullptr || (a->T > 0 && a->perm_idx == nullptr))
      return fail(MFR_ERR_INVALID_ARG, "the expert order needs perm_idx, row_route and expert_counts beside expert_offsets");
    const int64_t rows = moe_route_max_rows(a->T, a->K, a->E, a->row_align);
    if (rows < 0) return static_cast<int>(rows);
    if (a->num_rows < rows || a->num_rows > INT32_MAX)
      return fail(MFR_ERR_INVALID_ARG, "num_rows = %lld outside [moe_route_max_rows = %lld, 2^31)", static_cast<long long>(a->num_rows),
                  static_cast<long long>(rows));
    if (a->num_rows > 0 && a->row_route == nullptr) return fail(MFR_ERR_INVALID_ARG, "row_route is NULL");
    if (!aligned(a->perm_idx, 4) || !aligned(a->row_route, 4) || !aligned(a->expert_offsets, 4) || !aligned(a->expert_counts, 4))
      return fail(MFR_ERR_INVALID_ARG, "perm_idx, row_route, expert_offsets or expert_counts not 4-byte aligned");
    const int64_t need = moe_route_workspace_bytes(a->T, a->K, a->E);
    if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need || !aligned(a->workspace, 16)))
      return fail(MFR_ERR_INVALID_ARG, "the workspace must hold %lld bytes, 16-byte aligned", static_cast<long long>(need));
  } else if (a->perm_idx != nullptr || a->row_route != nullptr || a->expert_counts != nullptr) {
    return fail(MFR_ERR_INVALID_ARG, "perm_idx, row_route and expert_counts need expert_offsets");
  }
  if (!aligned(a->bias, 4)) return fail(MFR_ERR_INVALID_ARG, "bias not aligned to its type");  // (read without tokens too)
  if (a->T == 0) return MFR_OK;
  if (a->logits == nullptr || a->expert_ids == nullptr || a->expert_scale == nullptr)
    return fail(MFR_ERR_INVALID_ARG, "logits, expert_ids or expert_scale is NULL");
  if (!aligned(a->logits, dtype_bytes(a->logits_dtype)) || !aligned(a->expert_ids, 4) ||
      !aligned(a->expert_scale, dtype_bytes(a->scale_dtype)))
    return fail(MFR_ERR_INVALID_ARG, "logits, expert_ids or expert_scale not aligned to its type");
  return MFR_OK;
}

int check_route_backward(const mfr_route_backward_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_routes(a->T, a->K)) != MFR_OK || (st = check_experts(a->E, a->K)) != MFR_OK ||
      (st = check_scoring(a->logits_dtype, a->scale_dtype, a->score, a->renormalize)) != MFR_OK ||
      (st = check_flags(a->flags, MFR_FLAG_PDL)) != MFR_OK ||
      (st = check_stride("logits_stride", a->logits_stride, a->E)) != MFR_OK ||
      (st = check_stride("d_logits_stride", a->d_logits_stride, a->E)) != MFR_OK)
    return st;
  if (a->T == 0) return MFR_OK;
  if (a->logits == nullptr || a->expert_ids == nullptr || a->d_scale == nullptr || a->d_logits == nullptr)
    return fail(MFR_ERR_INVALID_ARG, "logits, expert_ids, d_scale or d_logits is NULL");
  const uintptr_t lb = dtype_bytes(a->logits_dtype);
  if (!aligned(a->logits, lb) || !aligned(a->d_logits, lb) || !aligned(a->expert_ids, 4) ||
      !aligned(a->d_scale, dtype_bytes(a->scale_dtype)))
    return fail(MFR_ERR_INVALID_ARG, "logits, d_logits, expert_ids or d_scale not aligned to its type");
  return MFR_OK;
}

int check_dispatch(const mfr_dispatch_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_routes(a->T, a->K)) != MFR_OK || (st = check_flags(a->flags, MFR_FLAG_PDL)) != MFR_OK) return st;
  if (a->row_bytes < 16 || a->row_bytes % 16 != 0 || a->row_bytes > (1 << 20))
    return fail(MFR_ERR_INVALID_ARG, "row_bytes = %lld must be a multiple of 16 in [16, 2^20]", static_cast<long long>(a->row_bytes));
  if (a->num_rows < 0 || a->num_rows > INT32_MAX) return fail(MFR_ERR_INVALID_ARG, "num_rows = %lld outside [0, 2^31)", static_cast<long long>(a->num_rows));
  if (a->T > 0 && (a->x == nullptr || a->perm_idx == nullptr)) return fail(MFR_ERR_INVALID_ARG, "x or perm_idx is NULL");
  if (a->num_rows > 0 && a->rows == nullptr) return fail(MFR_ERR_INVALID_ARG, "rows is NULL");
  if (!aligned(a->x, 16) || !aligned(a->rows, 16)) return fail(MFR_ERR_INVALID_ARG, "x or rows not 16-byte aligned");
  if (!aligned(a->perm_idx, 4) || !aligned(a->row_route, 4)) return fail(MFR_ERR_INVALID_ARG, "perm_idx or row_route not 4-byte aligned");
  return MFR_OK;
}

int check_routed_backward(const mfr_routed_backward_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_routes(a->T, a->K)) != MFR_OK || (st = check_flags(a->flags, MFR_FLAG_PDL)) != MFR_OK) return st;
  if (a->H < 8 || a->H > MFR_MAX_HIDDEN || a->H % 8 != 0)
    return fail(MFR_ERR_INVALID_ARG, "H = %d must be a multiple of 8 in [8, %d]", a->H, MFR_MAX_HIDDEN);
  if (a->act_dtype != MFR_BF16 && a->act_dtype != MFR_FP16)
    return fail(MFR_ERR_UNSUPPORTED, "act_dtype %d: only MFR_BF16 and MFR_FP16", a->act_dtype);
  if (!any_dtype(a->scale_dtype)) return fail(MFR_ERR_UNSUPPORTED, "scale_dtype %d unknown", a->scale_dtype);
  if (a->num_rows < 0 || a->num_rows > INT32_MAX) return fail(MFR_ERR_INVALID_ARG, "num_rows = %lld outside [0, 2^31)", static_cast<long long>(a->num_rows));
  if (a->d_gemm2 == nullptr && a->d_scale == nullptr) return fail(MFR_ERR_INVALID_ARG, "no output requested");
  if (a->d_scale != nullptr && a->num_rows > 0 && a->gemm2_out == nullptr)
    return fail(MFR_ERR_INVALID_ARG, "d_scale needs gemm2_out");
  if (a->T > 0 && (a->d_out == nullptr || a->perm_idx == nullptr)) return fail(MFR_ERR_INVALID_ARG, "d_out or perm_idx is NULL");
  if (!aligned(a->gemm2_out, 16) || !aligned(a->d_out, 16) || !aligned(a->d_gemm2, 16))
    return fail(MFR_ERR_INVALID_ARG, "gemm2_out, d_out or d_gemm2 not 16-byte aligned");
  const uintptr_t sb = dtype_bytes(a->scale_dtype);
  if (!aligned(a->perm_idx, 4) || !aligned(a->row_route, 4) || !aligned(a->expert_scale, sb) || !aligned(a->d_scale, sb))
    return fail(MFR_ERR_INVALID_ARG, "perm_idx, row_route, expert_scale or d_scale not aligned to its type");
  return MFR_OK;
}

// `D`: of an output, whose heads must not overlap one another; 0 for an input.
int check_heads(const char* name, const mfr_heads& h, int heads, int T, int D) {
  if (heads == 0 || T == 0) return MFR_OK;
  if (h.data == nullptr) return fail(MFR_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(h.data, 16) || h.token_stride % 8 != 0 || h.head_stride % 8 != 0)
    return fail(MFR_ERR_INVALID_ARG, "%s must start on 16 bytes, with strides of multiples of 8 elements", name);
  // far inside 64 bits: T and heads are below 2^31
  if (std::llabs(h.token_stride) > (int64_t{1} << 30) || std::llabs(h.head_stride) > (int64_t{1} << 30))
    return fail(MFR_ERR_INVALID_ARG, "%s: strides above 2^30", name);
  if ((T > 1 && std::llabs(h.token_stride) < D) || (heads > 1 && std::llabs(h.head_stride) < D))
    return fail(MFR_ERR_INVALID_ARG, "%s: heads or tokens closer than D = %d elements", name, D);
  return MFR_OK;
}

int check_head_norm(const mfr_head_norm_args* a, bool backward) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_flags(a->flags, MFR_FLAG_PDL | MFR_FLAG_ZERO_PADDING | MFR_FLAG_POSITIONS_64)) != MFR_OK) return st;
  if (a->T < 0) return fail(MFR_ERR_INVALID_ARG, "T = %d < 0", a->T);
  if (a->q_heads < 0 || a->k_heads < 0 || a->q_heads > kMaxHeads || a->k_heads > kMaxHeads || a->q_heads + a->k_heads == 0)
    return fail(MFR_ERR_INVALID_ARG, "q_heads = %d, k_heads = %d: each in [0, %d], not both 0", a->q_heads, a->k_heads, kMaxHeads);
  if (a->D < 16 || a->D > MFR_MAX_HEAD_DIM || a->D % 16 != 0)
    return fail(MFR_ERR_INVALID_ARG, "D = %d must be a multiple of 16 in [16, %d]", a->D, MFR_MAX_HEAD_DIM);
  if (a->style != MFR_ROTARY_HALF && a->style != MFR_ROTARY_INTERLEAVED)
    return fail(MFR_ERR_UNSUPPORTED, "style %d unknown", a->style);
  const int unit = a->style == MFR_ROTARY_HALF ? 16 : 2;
  if (a->rot < 0 || a->rot > a->D || a->rot % unit != 0)
    return fail(MFR_ERR_INVALID_ARG, "rot = %d must be a multiple of %d in [0, D = %d]", a->rot, unit, a->D);
  if (a->act_dtype != MFR_BF16 && a->act_dtype != MFR_FP16)
    return fail(MFR_ERR_UNSUPPORTED, "act_dtype %d: only MFR_BF16 and MFR_FP16", a->act_dtype);
  if ((st = check_heads("q", a->q, a->q_heads, a->T, 0)) != MFR_OK || (st = check_heads("k", a->k, a->k_heads, a->T, 0)) != MFR_OK ||
      (st = check_heads("q_out", a->q_out, a->q_heads, a->T, a->D)) != MFR_OK ||
      (st = check_heads("k_out", a->k_out, a->k_heads, a->T, a->D)) != MFR_OK)
    return st;
  if (backward && ((st = check_heads("d_q_out", a->d_q_out, a->q_heads, a->T, 0)) != MFR_OK ||
                   (st = check_heads("d_k_out", a->d_k_out, a->k_heads, a->T, 0)) != MFR_OK))
    return st;
  if (!aligned(a->q_weight, 16) || !aligned(a->k_weight, 16)) return fail(MFR_ERR_INVALID_ARG, "q_weight or k_weight not 16-byte aligned");
  if (!aligned(a->positions, (a->flags & MFR_FLAG_POSITIONS_64) ? 8 : 4) || !aligned(a->inv_freq, 4))
    return fail(MFR_ERR_INVALID_ARG, "positions or inv_freq not aligned to its type");
  if (a->T > 0 && a->positions == nullptr) return fail(MFR_ERR_INVALID_ARG, "positions is NULL");
  if (a->T > 0 && a->rot > 0 && a->inv_freq == nullptr) return fail(MFR_ERR_INVALID_ARG, "inv_freq is NULL");
  if (backward && (a->d_q_weight != nullptr || a->d_k_weight != nullptr)) {
    if (!aligned(a->d_q_weight, 4) || !aligned(a->d_k_weight, 4)) return fail(MFR_ERR_INVALID_ARG, "d_q_weight or d_k_weight not 4-byte aligned");
    const int64_t need = moe_head_norm_rotary_workspace_bytes(a->T, a->q_heads, a->k_heads, a->D);
    if (a->workspace == nullptr || a->workspace_bytes < need || !aligned(a->workspace, 16))
      return fail(MFR_ERR_INVALID_ARG, "the workspace must hold %lld bytes, 16-byte aligned", static_cast<long long>(need));
  }
  return MFR_OK;
}

}  // namespace
}  // namespace mfr

using namespace mfr;

extern "C" {

int moe_route(const mfr_route_args* args, struct CUstream_st* stream) {
  const int st = check_route(args);
  if (st != MFR_OK || (args->T == 0 && args->expert_offsets == nullptr)) return st;
  return enqueue_status(launch_route(*args, stream), "moe_route launch");
}

int64_t moe_route_max_rows(int32_t T, int32_t K, int32_t E, int32_t row_align) {
  int st;
  if ((st = check_routes(T, K)) != MFR_OK || (st = check_experts(E, K)) != MFR_OK) return st;
  if (row_align < 1) return fail(MFR_ERR_INVALID_ARG, "row_align = %d < 1", row_align);
  // every expert with routes adds at most row_align - 1 rows of padding, and the sum is a multiple of row_align
  const int64_t n = static_cast<int64_t>(T) * K;
  const int64_t rows = (n + (n < E ? n : E) * (row_align - 1)) / row_align * row_align;
  if (rows > INT32_MAX) return fail(MFR_ERR_INVALID_ARG, "%lld padded rows: 2^31 or more", static_cast<long long>(rows));
  return rows;
}

int64_t moe_route_workspace_bytes(int32_t T, int32_t K, int32_t E) {
  int st;
  if ((st = check_routes(T, K)) != MFR_OK || (st = check_experts(E, K)) != MFR_OK) return st;
  const int chunks = route_chunks(T, E, true);
  return chunks > kRouteCluster ? (static_cast<int64_t>(chunks) * E * 4 + 15) / 16 * 16 : 0;  // the chunks' counts of each expert
}

int moe_route_backward(const mfr_route_backward_args* args, struct CUstream_st* stream) {
  const int st = check_route_backward(args);
  if (st != MFR_OK || args->T == 0) return st;
  return enqueue_status(launch_route_backward(*args, stream), "moe_route_backward launch");
}

int moe_dispatch_rows(const mfr_dispatch_args* args, struct CUstream_st* stream) {
  const int st = check_dispatch(args);
  if (st != MFR_OK || args->num_rows == 0 || (args->T == 0 && args->row_route == nullptr)) return st;
  return enqueue_status(launch_dispatch(*args, stream), "moe_dispatch_rows launch");
}

int moe_routed_backward(const mfr_routed_backward_args* args, struct CUstream_st* stream) {
  const int st = check_routed_backward(args);
  if (st != MFR_OK) return st;
  const bool zeros = args->row_route != nullptr && args->d_gemm2 != nullptr && args->num_rows > 0;
  if (args->T == 0 && !zeros) return MFR_OK;
  return enqueue_status(launch_routed_backward(*args, stream), "moe_routed_backward launch");
}

int moe_head_norm_rotary(const mfr_head_norm_args* args, struct CUstream_st* stream) {
  const int st = check_head_norm(args, false);
  if (st != MFR_OK || args->T == 0) return st;
  return enqueue_status(launch_head_norm(*args, stream), "moe_head_norm_rotary launch");
}

int64_t moe_head_norm_rotary_workspace_bytes(int32_t T, int32_t q_heads, int32_t k_heads, int32_t D) {
  if (T < 0 || q_heads < 0 || k_heads < 0 || q_heads > kMaxHeads || k_heads > kMaxHeads || D < 16 || D > MFR_MAX_HEAD_DIM || D % 16 != 0)
    return fail(MFR_ERR_INVALID_ARG, "T >= 0, q_heads and k_heads in [0, %d] and D a multiple of 16 in [16, %d]", kMaxHeads, MFR_MAX_HEAD_DIM);
  return std::max(static_cast<int64_t>(head_grad_rows(T, q_heads, k_heads, D)) * 2 * D * 4, int64_t{16});
}

int moe_head_norm_rotary_backward(const mfr_head_norm_args* args, struct CUstream_st* stream) {
  const int st = check_head_norm(args, true);
  if (st != MFR_OK || (args->T == 0 && args->d_q_weight == nullptr && args->d_k_weight == nullptr)) return st;
  return enqueue_status(launch_head_norm_backward(*args, stream), "moe_head_norm_rotary_backward launch");
}

}  // extern "C"
