// Internal launch interface of the routed-expert operators: routing, the
// expert-sorted rows, MXFP4 quantisation and products, the weighted sum.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lora {

// A grid of `blocks` workgroups of 256 threads, and a workgroup's number in
// it. A launch takes fewer than 2^32 threads along one dimension: of more it
// runs the remainder modulo 2^32 and reports no error. So past 2^23 workgroups
// the grid has a second dimension, whose last row may be past `blocks`.
constexpr int64_t kGridX = (int64_t)1 << 23;
inline dim3 grid_of(int64_t blocks) {
  return dim3((unsigned)(blocks < kGridX ? blocks : kGridX),
              (unsigned)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ uint32_t block_of_grid() {
  return blockIdx.y * (uint32_t)kGridX + blockIdx.x;
}

// Scores, groups and weights of lora_route_experts (see the C ABI).
struct RouteArgs {
  int T, E, k;
  int sigmoid;       // scores: sigmoid, else softmax
  int groups, top_groups;
  int sum2;          // a group's worth: sum of its two best, else its best
  int renorm;
  float scaling;
};
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxGroups = 16;
hipError_t launch_route_experts(int dtype, const void* logits, const float* bias,
                                const RouteArgs& a, int32_t* ids, float* weights,
                                hipStream_t stream);

// Expert-sorted rows of T * k choices (lora_expert_rows): at most so many that
// a count rounded up to a block of 1024 is an int.
constexpr int64_t kMaxSortedChoices = ((int64_t)1 << 31) - 1024;
size_t expert_rows_workspace_bytes(int64_t T, int k, int E);
hipError_t launch_expert_rows(const int32_t* ids, int T, int k, int E, const int32_t* token_slot,
                              int32_t* row_token, int32_t* positions, int32_t* offsets,
                              int32_t* row_slot, void* ws, hipStream_t stream);

hipError_t launch_combine_experts(int dtype, const void* rows, int64_t nrows, int H,
                                  const int32_t* positions, const float* weights, int T, int k,
                                  const void* residual, void* y, hipStream_t stream);

// Bytes of a scale row of K values: K / 32, padded to a multiple of four.
inline int mx_scale_row(int64_t K) { return (int)((K / 32 + 3) & ~(int64_t)3); }

// form of the rows quantised
constexpr int kQuantPlain = 0, kQuantGather = 1, kQuantSiluMul = 2;
hipError_t launch_quantize_mxfp4(int dtype, int form, const void* x, int64_t src_rows,
                                 const int32_t* row_index, int64_t rows, int K, void* rows_out,
                                 uint8_t* codes, uint8_t* scales, hipStream_t stream);
hipError_t launch_dequantize_mxfp4(int dtype, const uint8_t* codes, const uint8_t* scales,
                                   int64_t rows, int K, void* out, hipStream_t stream);

// y[r] = x[r] @ w[e(r)]^T over MXFP4 operands. offsets == nullptr: one weight
// for every row (E = 1).
struct MxArgs {
  const uint8_t* x;
  const uint8_t* xs;
  const uint8_t* w;
  const uint8_t* ws;
  void* y;
  const int32_t* offsets;
  int rows, N, K, E;
};
hipError_t launch_mxfp4_linear(int dtype, const MxArgs& a, hipStream_t stream);

}  // namespace lora
