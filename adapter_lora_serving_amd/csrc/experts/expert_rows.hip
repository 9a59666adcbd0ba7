// The rows of the experts' products, and the way back to tokens.
//
// Page "spark_model/lora/expert_apply.rs" (module overview): the experts'
// products run on rows sorted by expert, each expert's rows between two of
// its offsets, and a reduction brings them back to tokens. expert_rows sorts
// the T * k (token, choice) pairs of a routed batch that way, on the device:
// the stable counting sort of the slot addressing with the expert as the key
// (a choice outside [0, E) is dead and comes after every expert), then each
// row's token, its token's adapter slot and each choice's row.
#include "lora_common.h"
#include "lora_kernels.h"
#include "experts.h"

namespace lora {

// row_token holds the sorted choices (token * k + j) on entry and the tokens
// on return; every thread turns its own.
__global__ __launch_bounds__(256) void k_rows_finish(int n, int k, int E,
                                                     const int32_t* __restrict__ offsets,
                                                     const int32_t* __restrict__ token_slot,
                                                     int32_t* row_token,
                                                     int32_t* __restrict__ positions,
                                                     int32_t* __restrict__ row_slot) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= n) return;
  const int choice = row_token[r];
  const int t = choice / k;
  const bool live = r < offsets[E];
  row_token[r] = t;
  positions[choice] = live ? r : -1;
  if (row_slot) row_slot[r] = live ? token_slot[t] : -1;
}

size_t expert_rows_workspace_bytes(int64_t T, int k, int E) {
  return addressing_workspace_bytes(T * k, E);
}

hipError_t launch_expert_rows(const int32_t* ids, int T, int k, int E, const int32_t* token_slot,
                              int32_t* row_token, int32_t* positions, int32_t* offsets,
                              int32_t* row_slot, void* ws, hipStream_t stream) {
  const int n = T * k;
  hipError_t e = launch_build_addressing(ids, n, E, row_token, offsets, ws,
                                         expert_rows_workspace_bytes(T, k, E), stream);
  if (e != hipSuccess || n == 0) return e;
  hipLaunchKernelGGL(k_rows_finish, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, n, k,
                     E, offsets, token_slot, row_token, positions, row_slot);
  return hipGetLastError();
}

// y[t] = residual[t] + sum over j of weights[t, j] * rows[positions[t, j]],
// j ascending in fp32, rounded once. A position outside [0, nrows) adds
// nothing. 8 (bf16) or 4 (f32) columns per thread.
template <typename D>
__global__ __launch_bounds__(256) void k_combine(const char* __restrict__ rows, int64_t nrows,
                                                 int H, const int32_t* __restrict__ positions,
                                                 const float* __restrict__ weights, int k,
                                                 const char* __restrict__ residual,
                                                 char* __restrict__ y) {
  const int t = blockIdx.x;
  const int64_t rowb = (int64_t)H * D::kBytes;
  for (int c = threadIdx.x * 16; c < rowb; c += 256 * 16) {
    float acc[D::kVec];
    auto add = [&](u32x4 v, float w) {
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D::kVec == 8) {
          acc[2 * i] += w * bf16lo(q[i]);
          acc[2 * i + 1] += w * bf16hi(q[i]);
        } else {
          acc[i] += w * __uint_as_float(q[i]);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) acc[i] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int p = positions[(int64_t)t * k + j];
      if (p < 0 || p >= nrows) continue;
      add(*(const u32x4*)(rows + p * rowb + c), weights[(int64_t)t * k + j]);
    }
    if (residual) add(*(const u32x4*)(residual + t * rowb + c), 1.0f);
    u32x4 o;
    if constexpr (D::kVec == 8)
      o = u32x4{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7])};
    else
      o = u32x4{__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                __float_as_uint(acc[3])};
    *(u32x4*)(y + t * rowb + c) = o;
  }
}

hipError_t launch_combine_experts(int dtype, const void* rows, int64_t nrows, int H,
                                  const int32_t* positions, const float* weights, int T, int k,
                                  const void* residual, void* y, hipStream_t stream) {
  if (T == 0) return hipSuccess;
#define GO(D)                                                                                 \
  hipLaunchKernelGGL(k_combine<D>, dim3((unsigned)T), dim3(256), 0, stream, (const char*)rows, \
                     nrows, H, positions, weights, k, (const char*)residual, (char*)y)
  if (dtype == 1) GO(BF16); else GO(F32);
#undef GO
  return hipGetLastError();
}

}  // namespace lora
