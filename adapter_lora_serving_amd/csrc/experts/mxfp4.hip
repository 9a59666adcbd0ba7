// MXFP4 quantisation and its inverse.
//
// Microscaling format with 4-bit elements: a block of 32 consecutive values
// of a row has one scale byte b, standing for 2^(b - 127) (255: not a
// number), and 32 codes: a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6
// (E2M1). Quantisation takes b = floor(log2(max |x|)) - 2 + 127, the largest
// element's exponent against that of 6, clamped to [0, 254] (0 for an
// all-zero block, 255 where a value is NaN or infinite), and rounds each
// x * 2^(127 - b) to the nearest element, ties to the even code; values past
// 6 become 6. The even element of a pair is the low half of its byte.
#include "lora_common.h"
#include "experts.h"

namespace lora {

namespace {

// value * 2^(127 - byte) as a 4-bit code
__device__ __forceinline__ uint32_t code_of(float v, int shift) {
  const float a = fminf(ldexpf(fabsf(v), shift), 8.0f);
  const float r = a < 2.0f ? rintf(2.0f * a) : a < 4.0f ? rintf(a) + 2.0f : rintf(0.5f * a) + 4.0f;
  return (uint32_t)fminf(r, 7.0f) | ((__float_as_uint(v) >> 28) & 8u);
}

__device__ __forceinline__ float value_of(uint32_t code, float scale) {
  const uint32_t m = code & 7u;
  const float v = m < 2u ? 0.5f * (float)m : (1.0f + 0.5f * (float)(m & 1u)) * (float)(1u << ((m >> 1) - 1u));
  return ((code & 8u) ? -v : v) * scale;
}

__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 255u ? __builtin_nanf("") : ldexpf(1.0f, (int)byte - 127);
}

template <typename D>
__device__ __forceinline__ void load8(const char* p, float* v) {
  if constexpr (D::kBytes == 2) {
    const u32x4 q = *(const u32x4*)p;
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[2 * i] = bf16lo(u[i]); v[2 * i + 1] = bf16hi(u[i]); }
  } else {
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  }
}

template <typename D>
__device__ __forceinline__ void store8(char* p, const float* v) {
  if constexpr (D::kBytes == 2) {
    *(u32x4*)p = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7])};
  } else {
    *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4*)(p + 16) = f32x4{v[4], v[5], v[6], v[7]};
  }
}

}  // namespace

// One thread per 8 values, the 4 threads of a block of 32 side by side.
template <typename D, int FORM>
__global__ __launch_bounds__(256) void k_quantize(const char* __restrict__ x, int64_t src_rows,
                                                  const int32_t* __restrict__ row_index,
                                                  int64_t rows, int K, char* __restrict__ rows_out,
                                                  uint8_t* __restrict__ codes,
                                                  uint8_t* __restrict__ scales, int sld) {
  const int per_row = sld * 4;   // chunks of 8 over a row and its padding blocks
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = i / per_row;
  if (r >= rows) return;
  const int c = (int)(i - r * per_row) * 8;
  if (c >= K) {   // a padding block of the scale row
    if (c % 32 == 0) scales[r * sld + c / 32] = 0;
    return;
  }
  float v[8];
  if constexpr (FORM == kQuantSiluMul) {
    float gate[8], up[8];
    const char* row = x + r * 2 * K * D::kBytes;
    load8<D>(row + (int64_t)c * D::kBytes, gate);
    load8<D>(row + (int64_t)(K + c) * D::kBytes, up);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = gate[j] / (1.0f + expf(-gate[j])) * up[j];
  } else {
    int64_t src = r;
    if constexpr (FORM == kQuantGather) src = min(max((int64_t)row_index[r], (int64_t)0), src_rows - 1);
    load8<D>(x + (src * K + c) * D::kBytes, v);
  }
  if constexpr (FORM != kQuantPlain) {
    store8<D>(rows_out + (r * K + c) * D::kBytes, v);
    if constexpr (D::kBytes == 2) {   // the codes are those of the rounded row
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(to_bf16_bits(v[j]) << 16);
    }
  }
  // magnitudes order as their bits do, and NaN and infinity come last
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2));
  int byte;
  if (top >= 0x7f800000u) byte = 255;
  else byte = max((int)(top >> 23) - 2, 0);   // a denormal maximum clamps to 0 too
  uint32_t out = 0;
  if (byte != 255) {
#pragma unroll
    for (int j = 0; j < 8; ++j) out |= code_of(v[j], 127 - byte) << (4 * j);
  }
  *(uint32_t*)(codes + (r * K + c) / 2) = out;
  if (c % 32 == 0) scales[r * sld + c / 32] = (uint8_t)byte;
}

hipError_t launch_quantize_mxfp4(int dtype, int form, const void* x, int64_t src_rows,
                                 const int32_t* row_index, int64_t rows, int K, void* rows_out,
                                 uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int sld = mx_scale_row(K);
  const int64_t blocks = (rows * sld * 4 + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
#define GO(D, F)                                                                               \
  hipLaunchKernelGGL((k_quantize<D, F>), dim3((unsigned)blocks), dim3(256), 0, stream,         \
                     (const char*)x, src_rows, row_index, rows, K, (char*)rows_out, codes, scales, sld)
#define BY_FORM(D)                                   \
  do {                                               \
    if (form == kQuantPlain) GO(D, kQuantPlain);     \
    else if (form == kQuantGather) GO(D, kQuantGather); \
    else GO(D, kQuantSiluMul);                       \
  } while (0)
  if (dtype == 1) BY_FORM(BF16); else BY_FORM(F32);
#undef BY_FORM
#undef GO
  return hipGetLastError();
}

// One thread per 8 values.
template <typename D>
__global__ __launch_bounds__(256) void k_dequantize(const uint8_t* __restrict__ codes,
                                                    const uint8_t* __restrict__ scales,
                                                    int64_t rows, int K, char* __restrict__ out,
                                                    int sld) {
  const int per_row = K / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = i / per_row;
  if (r >= rows) return;
  const int c = (int)(i - r * per_row) * 8;
  const float scale = scale_of(scales[r * sld + c / 32]);
  const uint32_t q = *(const uint32_t*)(codes + (r * K + c) / 2);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = value_of((q >> (4 * j)) & 15u, scale);
  store8<D>(out + (r * K + c) * D::kBytes, v);
}

hipError_t launch_dequantize_mxfp4(int dtype, const uint8_t* codes, const uint8_t* scales,
                                   int64_t rows, int K, void* out, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int64_t blocks = (rows * (K / 8) + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
#define GO(D)                                                                               \
  hipLaunchKernelGGL(k_dequantize<D>, dim3((unsigned)blocks), dim3(256), 0, stream, codes, scales, \
                     rows, K, (char*)out, mx_scale_row(K))
  if (dtype == 1) GO(BF16); else GO(F32);
#undef GO
  return hipGetLastError();
}

}  // namespace lora
