// C ABI of the routed-expert operators: argument validation on the host and
// kernel launches on the caller's stream, by the same rules as lora_api.cpp
// (nothing allocated, nothing synchronised, device data never read here).
#include "lora_mi355x.h"

#include <hip/hip_runtime.h>

#include "experts.h"

namespace {

constexpr int64_t kMaxI32 = 0x7fffffff;
constexpr int64_t kMaxWidth = 1 << 20;   // columns or K of an operand
// values of one quantisation: 2^31 threads of 8, with the scale row's padding
// (at most 3 blocks in 4)
constexpr int64_t kMaxValues = (int64_t)1 << 32;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dtype_ok(int dtype) { return dtype == LORA_F32 || dtype == LORA_BF16; }
lora_status hip_status(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_ERR_HIP; }

lora_status check_mx(int64_t rows, int64_t K) {
  if (rows < 0 || rows > kMaxI32 || K < 1) return LORA_ERR_INVALID_ARG;
  if (K > kMaxWidth) return LORA_ERR_UNSUPPORTED;
  if (K % 32 != 0) return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}

lora_status check_choices(int64_t T, int32_t top_k, int32_t num_experts) {
  if (T < 0) return LORA_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > lora::kMaxTopK || num_experts < 1 || num_experts > lora::kMaxExperts)
    return LORA_ERR_UNSUPPORTED;
  if (T > kMaxI32 / top_k) return LORA_ERR_INVALID_ARG;   // T * top_k may pass 64 bits
  return LORA_OK;
}

// The sort counts in blocks of 1024 choices, in 32 bits.
lora_status check_sorted_choices(int64_t T, int32_t top_k, int32_t num_experts) {
  const lora_status st = check_choices(T, top_k, num_experts);
  return st == LORA_OK && T * top_k > lora::kMaxSortedChoices ? LORA_ERR_INVALID_ARG : st;
}

lora_status linear_impl(int dtype, const uint8_t* x_codes, const uint8_t* x_scales, int64_t rows,
                        const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, int64_t K,
                        const int32_t* offsets, int32_t num_experts, void* y, void* stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  const lora_status st = check_mx(rows, K);
  if (st != LORA_OK) return st;
  if (N < 1) return LORA_ERR_INVALID_ARG;
  if (N > kMaxWidth || num_experts < 1 || num_experts > lora::kMaxExperts)
    return LORA_ERR_UNSUPPORTED;
  if (rows == 0) return LORA_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y) return LORA_ERR_INVALID_ARG;
  if (!aligned16(x_codes) || !aligned16(w_codes) || !aligned16(y) || !aligned4(x_scales) ||
      !aligned4(w_scales))
    return LORA_ERR_ALIGNMENT;
  lora::MxArgs a;
  a.x = x_codes;
  a.xs = x_scales;
  a.w = w_codes;
  a.ws = w_scales;
  a.y = y;
  a.offsets = offsets;
  a.rows = (int)rows;
  a.N = (int)N;
  a.K = (int)K;
  a.E = num_experts;
  return hip_status(lora::launch_mxfp4_linear(dtype, a, (hipStream_t)stream));
}

}  // namespace

extern "C" {

lora_status lora_route_experts(int dtype, const void* logits, int64_t T, int32_t num_experts,
                               int32_t top_k, int32_t scores, const float* bias, int32_t groups,
                               int32_t top_groups, int32_t group_score, int32_t renormalize,
                               float scaling, int32_t* ids, float* weights, void* stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  const lora_status st = check_choices(T, top_k, num_experts);
  if (st != LORA_OK) return st;
  if (scores != LORA_SCORES_SOFTMAX && scores != LORA_SCORES_SIGMOID) return LORA_ERR_INVALID_ARG;
  if (group_score != LORA_GROUP_MAX && group_score != LORA_GROUP_SUM2) return LORA_ERR_INVALID_ARG;
  if (groups < 1 || groups > lora::kMaxGroups) return LORA_ERR_UNSUPPORTED;
  if (num_experts % groups != 0 || top_groups < 1 || top_groups > groups)
    return LORA_ERR_INVALID_ARG;
  if (top_k > num_experts / groups * top_groups) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!logits || !ids || !weights) return LORA_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned4(bias)) return LORA_ERR_ALIGNMENT;
  lora::RouteArgs a;
  a.T = (int)T;
  a.E = num_experts;
  a.k = top_k;
  a.sigmoid = scores == LORA_SCORES_SIGMOID;
  a.groups = groups;
  a.top_groups = top_groups;
  a.sum2 = group_score == LORA_GROUP_SUM2;
  a.renorm = renormalize != 0;
  a.scaling = scaling;
  return hip_status(
      lora::launch_route_experts(dtype, logits, bias, a, ids, weights, (hipStream_t)stream));
}

size_t lora_expert_rows_workspace_bytes(int64_t T, int32_t top_k, int32_t num_experts) {
  if (check_sorted_choices(T, top_k, num_experts) != LORA_OK) return 0;
  return lora::expert_rows_workspace_bytes(T, top_k, num_experts);
}

lora_status lora_expert_rows(const int32_t* ids, int64_t T, int32_t top_k, int32_t num_experts,
                             const int32_t* token_slot, int32_t* row_token, int32_t* positions,
                             int32_t* offsets, int32_t* row_slot, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const lora_status st = check_sorted_choices(T, top_k, num_experts);
  if (st != LORA_OK) return st;
  if (!offsets) return LORA_ERR_INVALID_ARG;
  if (T > 0 && (!ids || !row_token || !positions)) return LORA_ERR_INVALID_ARG;
  if (T > 0 && (token_slot == nullptr) != (row_slot == nullptr)) return LORA_ERR_INVALID_ARG;
  const size_t need = lora_expert_rows_workspace_bytes(T, top_k, num_experts);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LORA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LORA_ERR_ALIGNMENT;
  return hip_status(lora::launch_expert_rows(ids, (int)T, top_k, num_experts, token_slot,
                                             row_token, positions, offsets, row_slot, workspace,
                                             (hipStream_t)stream));
}

lora_status lora_combine_experts(int dtype, const void* rows, int64_t num_rows, int64_t width,
                                 const int32_t* positions, const float* weights, int64_t T,
                                 int32_t top_k, const void* residual, void* y, void* stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  const lora_status st = check_choices(T, top_k, 1);
  if (st != LORA_OK) return st;
  if (num_rows < 0 || num_rows > kMaxI32 || width < 1) return LORA_ERR_INVALID_ARG;
  if (width > kMaxWidth) return LORA_ERR_UNSUPPORTED;
  if (width % (dtype == LORA_BF16 ? 8 : 4) != 0) return LORA_ERR_ALIGNMENT;
  if (T == 0) return LORA_OK;
  if ((num_rows > 0 && !rows) || !positions || !weights || !y) return LORA_ERR_INVALID_ARG;
  if (!aligned16(rows) || !aligned16(residual) || !aligned16(y)) return LORA_ERR_ALIGNMENT;
  return hip_status(lora::launch_combine_experts(dtype, rows, num_rows, (int)width, positions,
                                                 weights, (int)T, top_k, residual, y,
                                                 (hipStream_t)stream));
}

int64_t lora_mxfp4_scale_row_bytes(int64_t K) {
  return check_mx(0, K) == LORA_OK ? lora::mx_scale_row(K) : 0;
}

lora_status lora_quantize_mxfp4(int dtype, int32_t form, const void* x, int64_t x_rows,
                                const int32_t* row_index, int64_t rows, int64_t K, void* rows_out,
                                uint8_t* codes, uint8_t* scales, void* stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  if (form != LORA_QUANTIZE_PLAIN && form != LORA_QUANTIZE_GATHER &&
      form != LORA_QUANTIZE_SILU_MUL)
    return LORA_ERR_INVALID_ARG;
  const lora_status st = check_mx(rows, K);
  if (st != LORA_OK) return st;
  if (x_rows < 0 || x_rows > kMaxI32) return LORA_ERR_INVALID_ARG;
  if (rows * K > kMaxValues) return LORA_ERR_UNSUPPORTED;
  if (rows == 0) return LORA_OK;
  if (!x || !codes || !scales) return LORA_ERR_INVALID_ARG;
  if (form == LORA_QUANTIZE_GATHER ? (!row_index || x_rows < 1) : x_rows < rows)
    return LORA_ERR_INVALID_ARG;
  if (form != LORA_QUANTIZE_PLAIN && !rows_out) return LORA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned4(scales) || !aligned16(rows_out))
    return LORA_ERR_ALIGNMENT;
  return hip_status(lora::launch_quantize_mxfp4(dtype, form, x, x_rows, row_index, rows, (int)K,
                                                rows_out, codes, scales, (hipStream_t)stream));
}

lora_status lora_dequantize_mxfp4(int dtype, const uint8_t* codes, const uint8_t* scales,
                                  int64_t rows, int64_t K, void* out, void* stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  const lora_status st = check_mx(rows, K);
  if (st != LORA_OK) return st;
  if (rows * K > kMaxValues) return LORA_ERR_UNSUPPORTED;
  if (rows == 0) return LORA_OK;
  if (!codes || !scales || !out) return LORA_ERR_INVALID_ARG;
  if (!aligned16(codes) || !aligned4(scales) || !aligned16(out)) return LORA_ERR_ALIGNMENT;
  return hip_status(lora::launch_dequantize_mxfp4(dtype, codes, scales, rows, (int)K, out,
                                                  (hipStream_t)stream));
}

lora_status lora_mxfp4_linear(int dtype, const uint8_t* x_codes, const uint8_t* x_scales,
                              int64_t rows, const uint8_t* w_codes, const uint8_t* w_scales,
                              int64_t N, int64_t K, void* y, void* stream) {
  return linear_impl(dtype, x_codes, x_scales, rows, w_codes, w_scales, N, K, nullptr, 1, y,
                     stream);
}

lora_status lora_mxfp4_expert_linear(int dtype, const uint8_t* x_codes, const uint8_t* x_scales,
                                     int64_t rows, const uint8_t* w_codes,
                                     const uint8_t* w_scales, int64_t N, int64_t K,
                                     const int32_t* offsets, int32_t num_experts, void* y,
                                     void* stream) {
  if (rows > 0 && !offsets) return LORA_ERR_INVALID_ARG;
  return linear_impl(dtype, x_codes, x_scales, rows, w_codes, w_scales, N, K, offsets,
                     num_experts, y, stream);
}

}  // extern "C"
