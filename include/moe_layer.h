/*
 * moe_layer.h -- C ABI of the operators around the fused MoE finalize (libmoe_finalize.so, sm_103a).
 *
 * They are the steps a layer takes on either side of moe_finalize_fused:
 *
 *   moe_route                      router logits -> chosen experts, their weights, and the expert order of
 *                                  the routes (perm_idx and expert_scale as moe_finalize_fused reads them)
 *   moe_route_backward             gradient of the weights -> gradient of the logits
 *   moe_dispatch_rows              token rows -> the expert-sorted rows that the expert products read
 *   moe_routed_backward            gradient of the finalized output -> gradients of the expert rows and of
 *                                  the expert scales
 *   moe_head_norm_rotary           per-head RMSNorm of queries and keys and their position rotation, in one pass
 *   moe_head_norm_rotary_backward  its gradients
 *
 * The conventions are those of moe_finalize.h: device pointers on the current device owned by the caller,
 * no allocation and no synchronization inside, a negative status before anything is enqueued on error
 * (message by moe_finalize_last_error), work enqueued on `stream`, MFR_FLAG_PDL to launch with programmatic
 * dependent launch (every kernel waits for its predecessor before reading or writing anything).  Two calls
 * that may run at the same time must not share a workspace.  Outputs overlap no input and not each other, unless
 * a call says so.  All sums, products, softmax and norm
 * statistics are FP32 or wider; an output in a 16-bit type is rounded once, to nearest even.  Every result
 * is the same from run to run: no atomic changes the order of a sum.
 */
#ifndef MOE_LAYER_H_
#define MOE_LAYER_H_

#include "moe_finalize.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MFR_MAX_EXPERTS 1024
#define MFR_MAX_GROUPS 32
#define MFR_MAX_HEAD_DIM 512

/* ---------------------------------------------------------------------------------------------------- */
/* Routing to experts                                                                                     */
/* ---------------------------------------------------------------------------------------------------- */

typedef enum { MFR_SCORE_SOFTMAX = 0, MFR_SCORE_SIGMOID = 1 } mfr_score;
typedef enum {
  MFR_GROUP_MAX = 0, /* a group's score is its best choice score                                        */
  MFR_GROUP_TOP2 = 1 /* a group's score is the sum of its two best choice scores (its best where it has one) */
} mfr_group_score;

/* Per token t, over its logits x_e:
 *
 *   s_e = softmax(x)_e or sigmoid(x_e)                        the score
 *   c_e = s_e + bias_e                                        the choice score (without bias: ordered by x_e)
 *   keep the topk_groups best of num_groups equal groups of consecutive experts (num_groups 1: all)
 *   expert_ids[t, 0..K-1] = the K largest c_e of the kept groups, best first
 *   w_k = s_{id_k}, divided by their sum if renormalize;  expert_scale[t, k] = round(w_k * scale)
 *
 * Equal choice scores (and group scores) go to the lowest index.  The order is decided as if the choice
 * scores were computed in 64 bits: scores that FP32 cannot tell apart safely are computed again in FP64.
 * An expert whose logit is -inf or NaN, or whose choice score is -inf or NaN, cannot be taken and counts 0
 * in the softmax; a token that has fewer than K experts to take gets id -1, weight 0 and perm_idx -1 in the
 * remaining places, which moe_finalize_fused skips.  A logit of +inf shares the softmax equally with the
 * token's other +inf logits.
 *
 * The expert order (all four outputs, or none): the routes t*K+k sorted by expert id, stably, expert e's
 * rows starting at expert_offsets[e], a multiple of row_align.
 *   perm_idx[t, k]       the row of route t*K+k, -1 for an id of -1
 *   row_route[r]         the route of row r, -1 for a row of no route (padding, and the rows behind the last)
 *   expert_offsets[e]    e = 0..E; expert_offsets[E] is the end of the last expert's padded rows
 *   expert_counts[e]     the routes of expert e
 */
typedef struct {
  int32_t T;              /* tokens, >= 0                                                               */
  int32_t E;              /* experts, 1..MFR_MAX_EXPERTS                                                 */
  int32_t K;              /* experts per token, 1..min(E, MFR_MAX_TOP_K); T*K < 2^31                     */
  int32_t logits_dtype;   /* mfr_dtype                                                                  */
  int32_t scale_dtype;    /* mfr_dtype of expert_scale                                                   */
  int32_t score;          /* mfr_score                                                                  */
  int32_t num_groups;     /* 1..MFR_MAX_GROUPS, divides E                                                */
  int32_t topk_groups;    /* 1..num_groups                                                              */
  int32_t group_score;    /* mfr_group_score                                                            */
  int32_t renormalize;    /* 0 or 1                                                                     */
  int32_t row_align;      /* >= 1: an expert's rows start at a multiple of it                            */
  float scale;            /* multiplies every weight                                                    */
  const void* logits;     /* device [T, E], rows logits_stride elements apart                            */
  int64_t logits_stride;  /* >= E                                                                       */
  const float* bias;      /* device [E] FP32, or NULL                                                    */
  int32_t* expert_ids;    /* device [T, K]                                                              */
  void* expert_scale;     /* device [T, K] of scale_dtype                                                */
  int32_t* perm_idx;      /* device [T, K]                                                              */
  int32_t* row_route;     /* device [num_rows]                                                          */
  int64_t num_rows;       /* with the expert order: >= moe_route_max_rows(T, K, E, row_align), < 2^31    */
  int32_t* expert_offsets;/* device [E + 1], or NULL: no expert order                                    */
  int32_t* expert_counts; /* device [E]                                                                 */
  void* workspace;        /* device, 16-byte aligned, moe_route_workspace_bytes bytes (NULL when that is 0) */
  int64_t workspace_bytes;
  uint32_t flags;         /* MFR_FLAG_PDL                                                               */
} mfr_route_args;

int moe_route(const mfr_route_args* args, struct CUstream_st* stream);

/* The most rows that T*K routes fill when every expert's rows are padded to a multiple of row_align. <0 on bad input. */
int64_t moe_route_max_rows(int32_t T, int32_t K, int32_t E, int32_t row_align);

/* Workspace bytes of moe_route with the expert order (0 for small batches). <0 on bad input. */
int64_t moe_route_workspace_bytes(int32_t T, int32_t K, int32_t E);

/* d_logits = the gradient of sum(d_scale * w * scale) with the chosen experts held fixed; experts that
 * were not chosen get their softmax's share (softmax without renormalize) or 0.  Ids outside [0, E) are
 * skipped; their d_scale is not used, whatever it holds.  Every element of d_logits is written. */
typedef struct {
  int32_t T, E, K;
  int32_t logits_dtype;      /* of logits and d_logits                                                  */
  int32_t scale_dtype;       /* of d_scale                                                              */
  int32_t score;
  int32_t renormalize;
  float scale;
  const void* logits;        /* device [T, E], rows logits_stride elements apart                         */
  int64_t logits_stride;
  const int32_t* expert_ids; /* device [T, K], as moe_route wrote them                                   */
  const void* d_scale;       /* device [T, K]                                                           */
  void* d_logits;            /* device [T, E], rows d_logits_stride elements apart                       */
  int64_t d_logits_stride;
  uint32_t flags;
} mfr_route_backward_args;

int moe_route_backward(const mfr_route_backward_args* args, struct CUstream_st* stream);

/* ---------------------------------------------------------------------------------------------------- */
/* Rows into expert order, and the gradient of the finalize                                               */
/* ---------------------------------------------------------------------------------------------------- */

/* rows[perm_idx[t, k]] = x[t] for every route whose perm_idx lies in [0, num_rows); no two routes may name
 * the same row.  With row_route (perm_idx the other way round, as moe_route writes it), rows whose route is
 * negative are set to zero; without it they are left as they were.  Rows of any type, copied as bytes.  Its gradient to
 * x is moe_finalize_fused in finalize-only mode over the gradient rows, with expert_scale NULL and a factor of 1. */
typedef struct {
  int32_t T, K;              /* K in 1..MFR_MAX_TOP_K, T*K < 2^31                                        */
  int64_t row_bytes;         /* bytes of a row, a positive multiple of 16, <= 2^20                       */
  int64_t num_rows;          /* rows of `rows` and of row_route, < 2^31                                  */
  const void* x;             /* device [T, row_bytes], 16-byte aligned                                   */
  const int32_t* perm_idx;   /* device [T, K]                                                           */
  const int32_t* row_route;  /* device [num_rows], or NULL                                               */
  void* rows;                /* device [num_rows, row_bytes], 16-byte aligned                            */
  uint32_t flags;
} mfr_dispatch_args;

int moe_dispatch_rows(const mfr_dispatch_args* args, struct CUstream_st* stream);

/* The gradient of one partial's finalize (finalize-only mode; the residual and the RMSNorm of the fused call have no
 * gradient here), out[t] = rsf * sum_k scale[t,k] * row[perm[t,k]] (+ shared row),
 * given d_out:
 *   d_gemm2[perm[t,k]] = round_act((scale[t,k] * rsf) * d_out[t])
 *   d_scale[t,k]       = round(rsf * sum_h row[perm[t,k], h] * d_out[t, h])        0 for a skipped route
 * (the gradient of the shared row is d_out itself).  Routes outside [0, num_rows) are skipped; no two routes
 * may name the same row.  With row_route (perm_idx the other way round), rows of d_gemm2 whose route is
 * negative are set to zero; without it they are left as they were. */
typedef struct {
  int32_t T, H, K;           /* as in mfr_args                                                          */
  int32_t act_dtype;         /* of gemm2_out, d_out, d_gemm2                                             */
  int32_t scale_dtype;       /* of expert_scale and d_scale                                              */
  float routed_scaling_factor;
  int64_t num_rows;          /* < 2^31                                                                  */
  const void* gemm2_out;     /* device [num_rows, H]; may be NULL when d_scale is                        */
  const int32_t* perm_idx;   /* device [T, K]                                                           */
  const void* expert_scale;  /* device [T, K], or NULL: every scale is 1                                 */
  const int32_t* row_route;  /* device [num_rows], or NULL                                               */
  const void* d_out;         /* device [T, H]                                                           */
  void* d_gemm2;             /* device [num_rows, H], or NULL (not written)                              */
  void* d_scale;             /* device [T, K], or NULL (not written)                                     */
  uint32_t flags;
} mfr_routed_backward_args;

int moe_routed_backward(const mfr_routed_backward_args* args, struct CUstream_st* stream);

/* ---------------------------------------------------------------------------------------------------- */
/* Per-head RMSNorm and position rotation of queries and keys                                             */
/* ---------------------------------------------------------------------------------------------------- */

typedef enum {
  MFR_ROTARY_HALF = 0,       /* pairs (i, i + rot/2); rot a multiple of 16                                */
  MFR_ROTARY_INTERLEAVED = 1 /* pairs (2i, 2i + 1); rot even                                             */
} mfr_rotary_style;

enum {
  /* Write zeros in the output rows of tokens whose position is negative (default: left as they were). */
  MFR_FLAG_ZERO_PADDING = 4u,
  /* positions holds int64 (default int32). */
  MFR_FLAG_POSITIONS_64 = 8u
};

/* One tensor of heads: element (t, h, i) at data + t*token_stride + h*head_stride + i (strides in elements,
 * multiples of 8; data 16-byte aligned). */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} mfr_heads;

/* Per token and head, x its D elements, w the kind's weight (NULL: ones):
 *   v_i = x_i * rstd * w_i,  rstd = 1 / sqrt(sum x^2 / D + eps)
 *   pair j of the first rot elements turned by the angle position * inv_freq[j], times rotary_scale:
 *     (a, b) -> (a cos - b sin, b cos + a sin) * rotary_scale;   the other elements pass
 *   out = round_act(...)                                       one rounding, after the rotation
 * The angle is reduced by integer arithmetic modulo one turn, so that far positions lose nothing: to within 2^-33 of a
 * turn for 32-bit positions and 2^-47 for 64-bit ones, of which the nearest 2^-32 is taken; |inv_freq| < 2^20.  A token
 * whose position is negative is padding: its values do not matter, and its output rows are left as they were, or set to
 * zero under MFR_FLAG_ZERO_PADDING.  An output may be its own input, with equal
 * strides (in place); otherwise outputs overlap no input and not each other. */
typedef struct {
  int32_t T;                 /* tokens, >= 0                                                            */
  int32_t q_heads, k_heads;  /* >= 0, not both 0                                                         */
  int32_t D;                 /* elements of a head, a multiple of 16, <= MFR_MAX_HEAD_DIM                */
  int32_t rot;               /* rotated elements, 0 <= rot <= D                                          */
  int32_t style;             /* mfr_rotary_style                                                        */
  int32_t act_dtype;         /* MFR_BF16 or MFR_FP16, of q, k, their weights and outputs                  */
  float eps;
  float rotary_scale;
  mfr_heads q, k;            /* inputs                                                                  */
  mfr_heads q_out, k_out;    /* outputs (backward: d_q, d_k)                                             */
  mfr_heads d_q_out, d_k_out;/* backward only: gradients of the outputs                                  */
  const void* q_weight;      /* device [D] act, 16-byte aligned, or NULL                                 */
  const void* k_weight;
  const void* positions;     /* device [T] int32 (int64 under MFR_FLAG_POSITIONS_64)                     */
  const float* inv_freq;     /* device [rot / 2] FP32                                                    */
  float* d_q_weight;         /* backward only: device [D] FP32, or NULL (not written)                    */
  float* d_k_weight;
  void* workspace;           /* backward only: device, 16-byte aligned                                   */
  int64_t workspace_bytes;   /* moe_head_norm_rotary_workspace_bytes, when a weight gradient is asked    */
  uint32_t flags;
} mfr_head_norm_args;

int moe_head_norm_rotary(const mfr_head_norm_args* args, struct CUstream_st* stream);

/* With u = inverse rotation of d_out (times rotary_scale on the rotated elements), g = u * w:
 *   d_x = round_act(rstd * (g - x * rstd^2 * mean(g * x)))
 *   d_w_i = sum over tokens and heads of u_i * x_i * rstd            (FP32, a fixed order)
 * A padding token adds nothing to d_w, and its d_q and d_k rows are set to zero whatever the flags. */
int moe_head_norm_rotary_backward(const mfr_head_norm_args* args, struct CUstream_st* stream);

/* Workspace bytes of the backward pass when a weight gradient is asked. <0 on bad input. */
int64_t moe_head_norm_rotary_workspace_bytes(int32_t T, int32_t q_heads, int32_t k_heads, int32_t D);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H_ */
