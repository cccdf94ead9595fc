/*
 * moe_experts.h -- C ABI of the experts' products (libmoe_finalize.so, sm_103a): what stands between moe_dispatch_rows
 * and moe_finalize_fused.
 *
 *   moe_expert_matmul              rows in expert order times their experts' weights, with the gate of the first product
 *   moe_expert_matmul_backward     its gradients: of the rows and of the weights
 *   moe_swiglu_backward            gradient of the gate between the two products
 *   moe_nvfp4_quantize             rows or weights -> NVFP4 codes and block scales, as moe_finalize_fused writes them
 *   moe_nvfp4_dequantize           and back
 *   moe_expert_matmul_nvfp4        NVFP4 rows times NVFP4 weights
 *
 * The conventions are those of moe_layer.h.  Rows are in expert order as moe_route and moe_dispatch_rows leave them:
 * expert e has the rows expert_offsets[e] .. expert_offsets[e] + expert_counts[e] - 1 (without counts: up to
 * expert_offsets[e + 1]), any number of them, none included.  The other rows belong to no expert: they are not used,
 * whatever they hold, and their output rows are left as they were, or set to zero under MFR_FLAG_ZERO_PADDING.
 * Offsets and counts are device data: they are cut to [0, num_rows].  Experts come in the order of their rows and must not share any:
 * where they do, no row outside is touched and rows' products take no more tiles than num_rows rows fill, but what is written is not defined.
 *
 * Products are of the stored values, exactly, and summed in FP32 by the tensor cores; what is rounded to 16 bits is
 * rounded once.  Every result is the same from run to run.
 */
#ifndef MOE_EXPERTS_H_
#define MOE_EXPERTS_H_

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MFR_MAX_EXPERT_WIDTH 65536
#define MFR_MAX_EXPERT_ROWS 2147482624 /* 2^31 - 1024: rows of a product, in whole tiles of any kernel */

/* ---------------------------------------------------------------------------------------------------- */
/* 16-bit products                                                                                        */
/* ---------------------------------------------------------------------------------------------------- */

/* For a row r of expert e, over the n_in values of the row:
 *   y_n = sum_i rows[r, i] * weight[e, n, i]
 *   out[r, n] = round(y_n)                                          n < n_out
 * or, gated, with 2 * n_out weight rows an expert (the gate's, then the others'):
 *   out[r, n] = round(y_n / (1 + exp(-y_n)) * y_(n_out + n))        n < n_out
 *   gate_up[r, n] = round(y_n)                                      n < 2 * n_out, where gate_up is not NULL */
typedef struct {
  int32_t E;                     /* experts, 1..MFR_MAX_EXPERTS                                          */
  int32_t n_in, n_out;           /* multiples of 8, 8..MFR_MAX_EXPERT_WIDTH                              */
  int32_t act_dtype;             /* MFR_BF16 or MFR_FP16, of every tensor here                           */
  int32_t gated;                 /* 0 or 1                                                              */
  int64_t num_rows;              /* rows of `rows` and `out`, 0..MFR_MAX_EXPERT_ROWS                      */
  const void* rows;              /* device [num_rows, n_in], 16-byte aligned                             */
  int64_t rows_stride;           /* elements from row to row, a multiple of 8, >= n_in                    */
  const void* weight;            /* device [E, n_out or 2 * n_out, n_in], 16-byte aligned                 */
  int64_t weight_stride;         /* elements from weight row to weight row, a multiple of 8, >= n_in      */
  int64_t weight_expert_stride;  /* elements from expert to expert, a multiple of 8                      */
  const int32_t* expert_offsets; /* device [E + 1]                                                      */
  const int32_t* expert_counts;  /* device [E], or NULL                                                 */
  void* out;                     /* device [num_rows, n_out], 16-byte aligned                            */
  int64_t out_stride;            /* a multiple of 8, >= n_out                                            */
  void* gate_up;                 /* device [num_rows, 2 * n_out], 16-byte aligned, or NULL               */
  int64_t gate_up_stride;        /* a multiple of 8, >= 2 * n_out                                        */
  uint32_t flags;                /* MFR_FLAG_PDL, MFR_FLAG_ZERO_PADDING                                  */
} mfr_expert_matmul_args;

int moe_expert_matmul(const mfr_expert_matmul_args* args, struct CUstream_st* stream);

/* The gradients of the product without the gate, given that of its output:
 *   d_rows[r, i]      = round(sum_n d_out[r, n] * weight[e, n, i])
 *   d_weight[e, n, i] = round(sum over the rows r of e of d_out[r, n] * rows[r, i])      0 for an expert of no rows
 * With accumulate (FP32 only), d_weight gets the sum added to it (magnitudes below 2^-126 count as 0). */
typedef struct {
  int32_t E;
  int32_t n_in, n_out;
  int32_t act_dtype;             /* of rows, weight, d_out, d_rows                                       */
  int32_t d_weight_dtype;        /* act_dtype or MFR_FP32                                                */
  int32_t accumulate;            /* 0 or 1                                                              */
  int64_t num_rows;
  const void* rows;              /* device [num_rows, n_in]; may be NULL when d_weight is                 */
  int64_t rows_stride;
  const void* weight;            /* device [E, n_out, n_in]; may be NULL when d_rows is                   */
  int64_t weight_stride;
  int64_t weight_expert_stride;
  const void* d_out;             /* device [num_rows, n_out], 16-byte aligned                            */
  int64_t d_out_stride;          /* a multiple of 8, >= n_out                                            */
  const int32_t* expert_offsets;
  const int32_t* expert_counts;
  void* d_rows;                  /* device [num_rows, n_in], 16-byte aligned, or NULL (not written)      */
  int64_t d_rows_stride;
  void* d_weight;                /* device [E, n_out, n_in] without gaps, 16-byte aligned, or NULL (not written) */
  uint32_t flags;                /* MFR_FLAG_PDL, MFR_FLAG_ZERO_PADDING (of d_rows)                      */
} mfr_expert_matmul_backward_args;

int moe_expert_matmul_backward(const mfr_expert_matmul_backward_args* args, struct CUstream_st* stream);

/* The gradient of out = g / (1 + exp(-g)) * u, g and u the halves of a row of gate_up, given that of out:
 *   p = 1 / (1 + exp(-g));   d_g = round(d * u * p * (1 + g * (1 - p)));   d_u = round(d * g * p)
 * and out itself again, for the gradient of the second product's weights.  With row_route, rows whose route is negative
 * are not read and get zeros. */
typedef struct {
  int64_t num_rows;              /* 0 <= num_rows < 2^31                                                */
  int32_t F;                     /* values of a half, a multiple of 8, 8..MFR_MAX_EXPERT_WIDTH            */
  int32_t act_dtype;             /* MFR_BF16 or MFR_FP16                                                 */
  const void* gate_up;           /* device [num_rows, 2 * F], 16-byte aligned                            */
  int64_t gate_up_stride;        /* a multiple of 8, >= 2 * F                                            */
  const void* d_out;             /* device [num_rows, F]; may be NULL when d_gate_up is                   */
  int64_t d_out_stride;          /* a multiple of 8, >= F                                                */
  const int32_t* row_route;      /* device [num_rows], or NULL                                           */
  void* d_gate_up;               /* device [num_rows, 2 * F], or NULL (not written); may be gate_up       */
  int64_t d_gate_up_stride;
  void* out;                     /* device [num_rows, F], or NULL (not written); may be d_out             */
  int64_t out_stride;
  uint32_t flags;                /* MFR_FLAG_PDL                                                        */
} mfr_swiglu_backward_args;

int moe_swiglu_backward(const mfr_swiglu_backward_args* args, struct CUstream_st* stream);

/* ---------------------------------------------------------------------------------------------------- */
/* NVFP4                                                                                                  */
/* ---------------------------------------------------------------------------------------------------- */

/* Each block of 16 values x of a row, as moe_finalize_fused quantises (every operation in FP32, rounded to nearest even):
 *   sf = e4m3(max|x| / 6 * scale), at most 448;   code = e2m1(x * (scale / sf)), at most 6 (0 where sf is 0)
 * and back: x = round(code * (sf / scale)).  The even value of a pair is in the low half of its byte.  Block scales are
 * row-major or in tiles of 128 rows x 4 blocks; the bytes of a tile behind the last row or block are set to zero.
 * `matrices` matrices of `rows` rows each follow one another (1: one tensor of rows), each with tiles of its own. */
typedef struct {
  int32_t matrices;              /* >= 1                                                                */
  int64_t rows;                  /* rows of a matrix, >= 0; matrices * rows < 2^31                        */
  int32_t H;                     /* a multiple of 16, 16..MFR_MAX_EXPERT_WIDTH                            */
  int32_t act_dtype;             /* MFR_BF16 or MFR_FP16, of x                                           */
  int32_t sf_layout;             /* MFR_SF_ROW_MAJOR or MFR_SF_SWIZZLED_128x4                            */
  void* x;                       /* device [matrices * rows, H], 16-byte aligned (quantize: read; dequantize: written) */
  int64_t x_stride;              /* a multiple of 8, >= H                                                */
  const float* scale;            /* device, one value > 0                                                */
  const int32_t* row_route;      /* device [matrices * rows], or NULL: rows of a negative route are not read and get zero
                                    codes and scales (quantize), or zeros (dequantize)                   */
  void* codes;                   /* device [matrices * rows, H / 2], 8-byte aligned                      */
  void* sf;                      /* device, moe_nvfp4_sf_bytes bytes                                     */
  uint32_t flags;                /* MFR_FLAG_PDL                                                        */
} mfr_nvfp4_args;

int moe_nvfp4_quantize(const mfr_nvfp4_args* args, struct CUstream_st* stream);
int moe_nvfp4_dequantize(const mfr_nvfp4_args* args, struct CUstream_st* stream);

/* Bytes of the block scales. <0 on bad input. */
int64_t moe_nvfp4_sf_bytes(int32_t matrices, int64_t rows, int32_t H, int32_t sf_layout);

/* moe_expert_matmul over NVFP4 rows and weights: the values are code * sf, and y is multiplied by alpha[e] (the inverse of
 * the two global scales) before the gate and the rounding.  n_in is a multiple of 64; gated, n_out is one of 128. */
typedef struct {
  int32_t E;
  int32_t n_in, n_out;
  int32_t out_dtype;             /* MFR_BF16 or MFR_FP16                                                 */
  int32_t gated;
  int64_t num_rows;
  const void* codes;             /* device [num_rows, n_in / 2], 16-byte aligned                         */
  const void* sf;                /* device [num_rows, n_in / 16] row-major, 4-byte aligned               */
  const void* weight_codes;      /* device [E, n_out or 2 * n_out, n_in / 2], 16-byte aligned             */
  const void* weight_sf;         /* device, E times the tiles of one expert's weight rows, 16-byte aligned */
  const float* alpha;            /* device [E], or NULL: ones                                            */
  const int32_t* expert_offsets;
  const int32_t* expert_counts;
  void* out;                     /* device [num_rows, n_out], 16-byte aligned                            */
  int64_t out_stride;
  void* workspace;               /* device, 16-byte aligned, moe_expert_matmul_nvfp4_workspace_bytes bytes (NULL when that is 0) */
  int64_t workspace_bytes;
  uint32_t flags;                /* MFR_FLAG_PDL, MFR_FLAG_ZERO_PADDING                                  */
} mfr_expert_matmul_nvfp4_args;

int moe_expert_matmul_nvfp4(const mfr_expert_matmul_nvfp4_args* args, struct CUstream_st* stream);

/* Workspace bytes of moe_expert_matmul_nvfp4 (0 for few rows an expert). <0 on bad input. */
int64_t moe_expert_matmul_nvfp4_workspace_bytes(int32_t E, int64_t num_rows, int32_t n_in);

/* Waits of the products' kernels that ran out (about 2 s without a step of a reduction; none does unless something is broken) since
 * the last call, on the current device, which is synchronized: every stream's calls count.  A call with such a wait ends and leaves its
 * outputs unfinished.  Test hook: under MFR_FLAG_TEST_STREAM_TIMEOUT the products' waits for their operands run out. */
int moe_expert_read_timeouts(uint32_t* count);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H_ */
