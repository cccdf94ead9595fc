// Host-side launch interface between the C ABI of the experts' products (experts_api.cu) and their kernels.
#pragma once

#include "layer_launch.h"
#include "moe_experts.h"

namespace mfr {

cudaError_t launch_expert_matmul(const mfr_expert_matmul_args& a, cudaStream_t stream);
cudaError_t launch_expert_rows_grad(const mfr_expert_matmul_backward_args& a, cudaStream_t stream);
cudaError_t launch_expert_weight_grad(const mfr_expert_matmul_backward_args& a, cudaStream_t stream);
cudaError_t launch_swiglu_backward(const mfr_swiglu_backward_args& a, cudaStream_t stream);
cudaError_t launch_nvfp4_quantize(const mfr_nvfp4_args& a, cudaStream_t stream);
cudaError_t launch_nvfp4_dequantize(const mfr_nvfp4_args& a, cudaStream_t stream);
cudaError_t launch_expert_matmul_nvfp4(const mfr_expert_matmul_nvfp4_args& a, cudaStream_t stream);
cudaError_t read_expert_timeouts(unsigned int* count);
cudaError_t read_expert_nvfp4_timeouts(unsigned int* count);

// Rows of an operand that one CTA's tile spans, and the most tiles of a call (tile numbers are 32-bit).
constexpr int kExpertTileRows = 128;
constexpr int64_t kExpertMaxTiles = int64_t{1} << 31;

// The NVFP4 product of more than kNvfp4FewRows rows an expert takes tiles of kNvfp4Rows rows, whose scales a kernel before it puts
// in order: for each tile and 64 values of the reduction two blocks of 128 rows' scales.
// Measured, 64 experts of 4096 x 4096, gated: 24 rows each 100 us by the small tile and 131 by the large one; 32 rows 101 and
// 132; 48 rows (two small tiles an expert) 151 and 136.  Rows vary from expert to expert, so the border is below 32.  R is the
// buffer's rows, so a decode step in a buffer aligned to 128 goes by the large tile: 16 tokens of 256 experts, top-8, 7168 x 2048 gated
// 171 us, where aligned to 8 or not at all it takes 117.
constexpr int kNvfp4FewRows = 24;
constexpr int kNvfp4Rows = 192;
inline bool nvfp4_few_rows(int64_t R, int E) { return R <= int64_t{kNvfp4FewRows} * E; }

// Tiles of `tile` rows that R rows of E experts fill at most.
inline int64_t expert_row_tiles(int64_t R, int E, int tile) { return R / tile + (R < E ? R : E); }

}  // namespace mfr
