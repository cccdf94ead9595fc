// C ABI of the experts' products (moe_experts.h): argument validation (nothing is enqueued on error), size queries and
// dispatch to the kernels.
#include <climits>
#include <mutex>

#include "experts_launch.h"
#include "mfr_launch.h"

namespace mfr {
namespace {

using ll = long long;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool act(int d) { return d == MFR_BF16 || d == MFR_FP16; }

int enqueue_status(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(MFR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return MFR_OK;
}

int check_flags(uint32_t flags, uint32_t known) {
  if (flags & ~known) return fail(MFR_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags & ~known);
  return MFR_OK;
}

int check_width(const char* name, int n, int unit) {
  if (n < unit || n > MFR_MAX_EXPERT_WIDTH || n % unit != 0)
    return fail(MFR_ERR_INVALID_ARG, "%s = %d must be a multiple of %d in [%d, %d]", name, n, unit, unit, MFR_MAX_EXPERT_WIDTH);
  return MFR_OK;
}

int check_rows(int64_t rows) {
  if (rows < 0 || rows > INT32_MAX) return fail(MFR_ERR_INVALID_ARG, "num_rows = %lld outside [0, 2^31)", static_cast<ll>(rows));
  return MFR_OK;
}

// Rows in expert order: the kernels round their numbers up to whole tiles in 32 bits.
int check_expert_rows(int64_t rows) {
  if (rows < 0 || rows > MFR_MAX_EXPERT_ROWS)
    return fail(MFR_ERR_INVALID_ARG, "num_rows = %lld outside [0, %lld]", static_cast<ll>(rows), static_cast<ll>(MFR_MAX_EXPERT_ROWS));
  return MFR_OK;
}

// A tensor of rows: its pointer and the distance of its rows in elements.
int check_tensor(const char* name, const void* p, int64_t stride, int64_t width) {
  if (p == nullptr || !aligned(p, 16)) return fail(MFR_ERR_INVALID_ARG, "%s is NULL or not 16-byte aligned", name);
  if (stride < width || stride % 8 != 0 || stride > (int64_t{1} << 31))
    return fail(MFR_ERR_INVALID_ARG, "%s: rows %lld elements apart; a multiple of 8 in [%lld, 2^31] is wanted", name, static_cast<ll>(stride),
                static_cast<ll>(width));
  return MFR_OK;
}

int check_experts(int E, int64_t num_rows, const int32_t* offsets, const int32_t* counts) {
  if (E < 1 || E > MFR_MAX_EXPERTS) return fail(MFR_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, MFR_MAX_EXPERTS);
  const int st = check_expert_rows(num_rows);
  if (st != MFR_OK) return st;
  if (offsets == nullptr || !aligned(offsets, 4) || !aligned(counts, 4))
    return fail(MFR_ERR_INVALID_ARG, "expert_offsets is NULL, or it or expert_counts not 4-byte aligned");
  return MFR_OK;
}

// Tile numbers are 32-bit.
int check_tiles(int64_t tiles) {
  if (tiles >= kExpertMaxTiles) return fail(MFR_ERR_INVALID_ARG, "%lld tiles: 2^31 or more", static_cast<ll>(tiles));
  return MFR_OK;
}
// The most tiles of any kernel for `rows` rows and `width` values a row.
int64_t row_tiles(int64_t rows, int E, int64_t width) { return expert_row_tiles(rows, E, kExpertTileRows) * ((width + 63) / 64); }

int check_weight(const void* p, int64_t stride, int64_t expert_stride, int E, int64_t rows, int64_t width) {
  const int st = check_tensor("weight", p, stride, width);
  if (st != MFR_OK) return st;
  if (E > 1 && (expert_stride % 8 != 0 || expert_stride < (rows - 1) * stride + width || expert_stride > (int64_t{1} << 38)))
    return fail(MFR_ERR_INVALID_ARG, "weight: experts %lld elements apart; a multiple of 8 that holds an expert, at most 2^38, is wanted",
                static_cast<ll>(expert_stride));
  return MFR_OK;
}

int check_matmul(const mfr_expert_matmul_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_experts(a->E, a->num_rows, a->expert_offsets, a->expert_counts)) != MFR_OK || (st = check_width("n_in", a->n_in, 8)) != MFR_OK ||
      (st = check_width("n_out", a->n_out, 8)) != MFR_OK || (st = check_flags(a->flags, MFR_FLAG_PDL | MFR_FLAG_ZERO_PADDING | MFR_FLAG_TEST_STREAM_TIMEOUT)) != MFR_OK)
    return st;
  if (!act(a->act_dtype)) return fail(MFR_ERR_UNSUPPORTED, "act_dtype %d: only MFR_BF16 and MFR_FP16", a->act_dtype);
  if (a->gated != 0 && a->gated != 1) return fail(MFR_ERR_INVALID_ARG, "gated = %d is not 0 or 1", a->gated);
  if (!a->gated && a->gate_up != nullptr) return fail(MFR_ERR_INVALID_ARG, "gate_up needs gated");
  const int64_t wide = a->gated ? int64_t{2} * a->n_out : a->n_out;
  if ((st = check_tiles(row_tiles(a->num_rows, a->E, wide))) != MFR_OK) return st;
  if (a->num_rows == 0) return MFR_OK;
  if ((st = check_tensor("rows", a->rows, a->rows_stride, a->n_in)) != MFR_OK ||
      (st = check_weight(a->weight, a->weight_stride, a->weight_expert_stride, a->E, wide, a->n_in)) != MFR_OK ||
      (st = check_tensor("out", a->out, a->out_stride, a->n_out)) != MFR_OK)
    return st;
  return a->gate_up == nullptr ? MFR_OK : check_tensor("gate_up", a->gate_up, a->gate_up_stride, wide);
}

int check_matmul_backward(const mfr_expert_matmul_backward_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_experts(a->E, a->num_rows, a->expert_offsets, a->expert_counts)) != MFR_OK || (st = check_width("n_in", a->n_in, 8)) != MFR_OK ||
      (st = check_width("n_out", a->n_out, 8)) != MFR_OK || (st = check_flags(a->flags, MFR_FLAG_PDL | MFR_FLAG_ZERO_PADDING | MFR_FLAG_TEST_STREAM_TIMEOUT)) != MFR_OK)
    return st;
  if (!act(a->act_dtype)) return fail(MFR_ERR_UNSUPPORTED, "act_dtype %d: only MFR_BF16 and MFR_FP16", a->act_dtype);
  if (a->d_weight_dtype != a->act_dtype && a->d_weight_dtype != MFR_FP32)
    return fail(MFR_ERR_UNSUPPORTED, "d_weight_dtype %d: act_dtype or MFR_FP32", a->d_weight_dtype);
  if (a->accumulate != 0 && a->accumulate != 1) return fail(MFR_ERR_INVALID_ARG, "accumulate = %d is not 0 or 1", a->accumulate);
  if (a->accumulate && a->d_weight_dtype != MFR_FP32) return fail(MFR_ERR_INVALID_ARG, "accumulate needs a d_weight in FP32");
  if (a->d_rows == nullptr && a->d_weight == nullptr) return fail(MFR_ERR_INVALID_ARG, "no output requested");
  if (!aligned(a->d_weight, 16)) return fail(MFR_ERR_INVALID_ARG, "d_weight not 16-byte aligned");
  if ((st = check_tiles(row_tiles(a->num_rows, a->E, a->n_in))) != MFR_OK ||
      (st = check_tiles(static_cast<int64_t>(a->E) * ((a->n_out + 127) / 128) * ((a->n_in + 63) / 64))) != MFR_OK)
    return st;
  if (a->num_rows == 0) return MFR_OK;
  if ((st = check_tensor("d_out", a->d_out, a->d_out_stride, a->n_out)) != MFR_OK) return st;
  if (a->d_rows != nullptr && ((st = check_tensor("d_rows", a->d_rows, a->d_rows_stride, a->n_in)) != MFR_OK ||
                               (st = check_weight(a->weight, a->weight_stride, a->weight_expert_stride, a->E, a->n_out, a->n_in)) != MFR_OK))
    return st;
  return a->d_weight == nullptr ? MFR_OK : check_tensor("rows", a->rows, a->rows_stride, a->n_in);
}

int check_swiglu_backward(const mfr_swiglu_backward_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_rows(a->num_rows)) != MFR_OK || (st = check_width("F", a->F, 8)) != MFR_OK || (st = check_flags(a->flags, MFR_FLAG_PDL)) != MFR_OK)
    return st;
  if (!act(a->act_dtype)) return fail(MFR_ERR_UNSUPPORTED, "act_dtype %d: only MFR_BF16 and MFR_FP16", a->act_dtype);
  if (a->d_gate_up == nullptr && a->out == nullptr) return fail(MFR_ERR_INVALID_ARG, "no output requested");
  if (!aligned(a->row_route, 4)) return fail(MFR_ERR_INVALID_ARG, "row_route not 4-byte aligned");
  if (a->num_rows == 0) return MFR_OK;
  const int64_t F = a->F;
  if ((st = check_tensor("gate_up", a->gate_up, a->gate_up_stride, 2 * F)) != MFR_OK) return st;
  if (a->d_gate_up != nullptr && ((st = check_tensor("d_gate_up", a->d_gate_up, a->d_gate_up_stride, 2 * F)) != MFR_OK ||
                                  (st = check_tensor("d_out", a->d_out, a->d_out_stride, F)) != MFR_OK))
    return st;
  return a->out == nullptr ? MFR_OK : check_tensor("out", a->out, a->out_stride, F);
}

int check_layout(int layout) {
  if (layout != MFR_SF_ROW_MAJOR && layout != MFR_SF_SWIZZLED_128x4) return fail(MFR_ERR_UNSUPPORTED, "sf_layout %d unknown", layout);
  return MFR_OK;
}

int check_matrices(int matrices, int64_t rows) {
  if (matrices < 1 || rows < 0 || rows > INT32_MAX || rows * matrices > INT32_MAX)
    return fail(MFR_ERR_INVALID_ARG, "matrices = %d >= 1 of rows = %lld >= 0, fewer than 2^31 in all, are wanted", matrices, static_cast<ll>(rows));
  return MFR_OK;
}

int check_nvfp4(const mfr_nvfp4_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_matrices(a->matrices, a->rows)) != MFR_OK || (st = check_width("H", a->H, 16)) != MFR_OK ||
      (st = check_layout(a->sf_layout)) != MFR_OK || (st = check_flags(a->flags, MFR_FLAG_PDL)) != MFR_OK)
    return st;
  // (a row of threads for each row of the tiles)
  if ((a->rows + 127) / 128 * 128 * a->matrices > INT32_MAX) return fail(MFR_ERR_INVALID_ARG, "rows in whole tiles: 2^31 or more");
  if (!act(a->act_dtype)) return fail(MFR_ERR_UNSUPPORTED, "act_dtype %d: only MFR_BF16 and MFR_FP16", a->act_dtype);
  if (a->scale == nullptr || !aligned(a->scale, 4) || !aligned(a->row_route, 4))
    return fail(MFR_ERR_INVALID_ARG, "scale is NULL, or it or row_route not 4-byte aligned");
  if (a->rows == 0) return MFR_OK;
  if ((st = check_tensor("x", a->x, a->x_stride, a->H)) != MFR_OK) return st;
  if (a->codes == nullptr || a->sf == nullptr || !aligned(a->codes, 8) || (a->sf_layout != MFR_SF_ROW_MAJOR && !aligned(a->sf, 16)))
    return fail(MFR_ERR_INVALID_ARG, "codes or sf is NULL, codes not 8-byte aligned or tiles of scales not 16-byte aligned");
  return MFR_OK;
}

int check_matmul_nvfp4(const mfr_expert_matmul_nvfp4_args* a) {
  if (a == nullptr) return fail(MFR_ERR_INVALID_ARG, "args is NULL");
  int st;
  if ((st = check_experts(a->E, a->num_rows, a->expert_offsets, a->expert_counts)) != MFR_OK || (st = check_width("n_in", a->n_in, 64)) != MFR_OK ||
      (st = check_width("n_out", a->n_out, a->gated == 1 ? 128 : 8)) != MFR_OK ||
      (st = check_flags(a->flags, MFR_FLAG_PDL | MFR_FLAG_ZERO_PADDING | MFR_FLAG_TEST_STREAM_TIMEOUT)) != MFR_OK)
    return st;
  if (!act(a->out_dtype)) return fail(MFR_ERR_UNSUPPORTED, "out_dtype %d: only MFR_BF16 and MFR_FP16", a->out_dtype);
  if (a->gated != 0 && a->gated != 1) return fail(MFR_ERR_INVALID_ARG, "gated = %d is not 0 or 1", a->gated);
  if ((st = check_tiles(row_tiles(a->num_rows, a->E, a->gated ? int64_t{2} * a->n_out : a->n_out))) != MFR_OK) return st;
  if (!aligned(a->alpha, 4)) return fail(MFR_ERR_INVALID_ARG, "alpha not 4-byte aligned");
  if (a->num_rows == 0) return MFR_OK;
  if (a->codes == nullptr || a->weight_codes == nullptr || !aligned(a->codes, 16) || !aligned(a->weight_codes, 16))
    return fail(MFR_ERR_INVALID_ARG, "codes or weight_codes is NULL or not 16-byte aligned");
  const int64_t need = moe_expert_matmul_nvfp4_workspace_bytes(a->E, a->num_rows, a->n_in);
  if (need < 0) return static_cast<int>(need);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need || !aligned(a->workspace, 16)))
    return fail(MFR_ERR_INVALID_ARG, "the workspace must hold %lld bytes, 16-byte aligned", static_cast<ll>(need));
  if (a->sf == nullptr || a->weight_sf == nullptr || !aligned(a->sf, 4) || !aligned(a->weight_sf, 16))
    return fail(MFR_ERR_INVALID_ARG, "sf or weight_sf is NULL, sf not 4-byte or weight_sf not 16-byte aligned");
  return check_tensor("out", a->out, a->out_stride, a->n_out);
}

}  // namespace
}  // namespace mfr

using namespace mfr;

extern "C" {

int moe_expert_matmul(const mfr_expert_matmul_args* args, struct CUstream_st* stream) {
  const int st = check_matmul(args);
  if (st != MFR_OK || args->num_rows == 0) return st;
  return enqueue_status(launch_expert_matmul(*args, stream), "moe_expert_matmul launch");
}

int moe_expert_matmul_backward(const mfr_expert_matmul_backward_args* args, struct CUstream_st* stream) {
  const int st = check_matmul_backward(args);
  if (st != MFR_OK) return st;
  if (args->d_rows != nullptr && args->num_rows > 0) {
    const int rc = enqueue_status(launch_expert_rows_grad(*args, stream), "moe_expert_matmul_backward launch (rows)");
    if (rc != MFR_OK) return rc;
  }
  if (args->d_weight == nullptr) return MFR_OK;
  return enqueue_status(launch_expert_weight_grad(*args, stream), "moe_expert_matmul_backward launch (weights)");
}

int moe_swiglu_backward(const mfr_swiglu_backward_args* args, struct CUstream_st* stream) {
  const int st = check_swiglu_backward(args);
  if (st != MFR_OK || args->num_rows == 0) return st;
  return enqueue_status(launch_swiglu_backward(*args, stream), "moe_swiglu_backward launch");
}

int64_t moe_nvfp4_sf_bytes(int32_t matrices, int64_t rows, int32_t H, int32_t sf_layout) {
  int st;
  if ((st = check_matrices(matrices, rows)) != MFR_OK || (st = check_width("H", H, 16)) != MFR_OK || (st = check_layout(sf_layout)) != MFR_OK) return st;
  const int64_t blocks = H / 16;
  return matrices * (sf_layout == MFR_SF_ROW_MAJOR ? rows * blocks : (rows + 127) / 128 * 128 * ((blocks + 3) / 4 * 4));
}

int moe_nvfp4_quantize(const mfr_nvfp4_args* args, struct CUstream_st* stream) {
  const int st = check_nvfp4(args);
  if (st != MFR_OK || args->rows == 0) return st;
  return enqueue_status(launch_nvfp4_quantize(*args, stream), "moe_nvfp4_quantize launch");
}

int moe_nvfp4_dequantize(const mfr_nvfp4_args* args, struct CUstream_st* stream) {
  const int st = check_nvfp4(args);
  if (st != MFR_OK || args->rows == 0) return st;
  return enqueue_status(launch_nvfp4_dequantize(*args, stream), "moe_nvfp4_dequantize launch");
}

int64_t moe_expert_matmul_nvfp4_workspace_bytes(int32_t E, int64_t num_rows, int32_t n_in) {
  int st;
  if (E < 1 || E > MFR_MAX_EXPERTS) return fail(MFR_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, MFR_MAX_EXPERTS);
  if ((st = check_expert_rows(num_rows)) != MFR_OK || (st = check_width("n_in", n_in, 64)) != MFR_OK) return st;
  if (nvfp4_few_rows(num_rows, E)) return 0;
  const int64_t blocks = expert_row_tiles(num_rows, E, kNvfp4Rows) * (n_in / 64) * 2;
  if (blocks > INT32_MAX) return fail(MFR_ERR_INVALID_ARG, "%lld blocks of scales: 2^31 or more", static_cast<ll>(blocks));
  return blocks * 512;
}

int moe_expert_matmul_nvfp4(const mfr_expert_matmul_nvfp4_args* args, struct CUstream_st* stream) {
  const int st = check_matmul_nvfp4(args);
  if (st != MFR_OK || args->num_rows == 0) return st;
  return enqueue_status(launch_expert_matmul_nvfp4(*args, stream), "moe_expert_matmul_nvfp4 launch");
}

int moe_expert_read_timeouts(uint32_t* count) {
  if (count == nullptr) return fail(MFR_ERR_INVALID_ARG, "count is NULL");
  // The device's counters only grow, so that no wait of a running kernel is lost; what was read last is kept here.
  constexpr int kDevices = 64;
  static std::mutex lock;
  static uint32_t known[kDevices] = {};
  const std::lock_guard<std::mutex> hold(lock);
  int dev = 0;
  unsigned int c = 0, q = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev >= kDevices) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();  // (the copies below wait for no stream that does not block)
  if (e == cudaSuccess) e = read_expert_timeouts(&c);
  if (e == cudaSuccess) e = read_expert_nvfp4_timeouts(&q);
  if (e != cudaSuccess) return fail(MFR_ERR_CUDA, "reading the timeout counters: %s", cudaGetErrorString(e));
  const uint32_t all = c + q;
  *count = all >= known[dev] ? all - known[dev] : all;  // (fewer: the device was reset)
  known[dev] = all;
  return MFR_OK;
}

}  // extern "C"
