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
//
// Bytes bound both ways: 8192 x 14336 bf16 from gate/up (470 MB in, 298 out)
// 155 us, 4.9 TB/s; back to bf16 (62 MB in, 235 out) 53 us, 5.6 TB/s. Sums are
// not involved; the activation is formed in fp32 and rounded to the rows' type
// once, and the codes are those of the rounded rows, so that quantising the
// rows gives the same codes.
#include "lora_common.h"
#include "experts.h"

namespace lora {

namespace {

// n / d for n < 2^31 as a product: mul = ceil(2^(31 + l) / d), l = ceil(log2 d),
// is below 2^32 and exact over that range. A 64-bit division a thread cost
// these kernels as much as their memory traffic.
struct Divider {
  uint32_t mul, shift, d;
};
Divider divider(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return Divider{(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l, d};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divider& v) {
  return (uint32_t)(((uint64_t)n * v.mul) >> v.shift);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight values / 2^(byte - 127) as 4-bit codes, the first in the low bits.
// v_cvt_scalef32_pk_fp4_f32 divides by the power of two, rounds to the
// nearest code, ties to the even one, and saturates (checked for every bf16
// value and every midpoint at every scale).
__device__ __forceinline__ uint32_t codes_of(const float* v, float scale) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
}

// 2^(byte - 127), byte 255: not a number. Byte 0 is 2^-127, a denormal.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23);
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

// v of the lane d = 1 or 2 away in its group of four.
template <int D>
__device__ __forceinline__ uint32_t quad_xor(uint32_t v) {
  constexpr int kPerm = D == 1 ? 0xb1 : 0x4e;   // lanes (1, 0, 3, 2) and (2, 3, 0, 1)
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kPerm, 0xf, 0xf, false);
}

}  // namespace

// One thread per 8 values, the 4 threads of a block of 32 side by side.
template <typename D, int FORM>
__global__ __launch_bounds__(256) void k_quantize(const char* __restrict__ x, int64_t src_rows,
                                                  const int32_t* __restrict__ row_index,
                                                  uint32_t chunks, Divider per_row, int K,
                                                  char* __restrict__ rows_out,
                                                  uint8_t* __restrict__ codes,
                                                  uint8_t* __restrict__ scales, int sld) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const uint32_t row = divide(i, per_row);
  const int64_t r = row;
  const int c = (int)(i - row * per_row.d) * 8;
  if (c >= K) {   // a padding block of the scale row
    if (c % 32 == 0) scales[r * sld + c / 32] = 0;
    return;
  }
  float v[8];
  if constexpr (FORM == kQuantSiluMul) {
    float gate[8], up[8];
    const char* src = x + r * 2 * K * D::kBytes;
    load8<D>(src + (int64_t)c * D::kBytes, gate);
    load8<D>(src + (int64_t)(K + c) * D::kBytes, up);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = gate[j] / (1.0f + expf(-gate[j])) * up[j];
  } else {
    int64_t src = r;
    if constexpr (FORM == kQuantGather)
      src = min(max((int64_t)row_index[r], (int64_t)0), src_rows - 1);
    load8<D>(x + (src * K + c) * D::kBytes, v);
  }
  if constexpr (FORM != kQuantPlain) {
    store8<D>(rows_out + (r * K + c) * D::kBytes, v);
    if constexpr (FORM == kQuantSiluMul && D::kBytes == 2) {   // the codes are those of the rounded row
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(to_bf16_bits(v[j]) << 16);
    }
  }
  // magnitudes order as their bits do, and NaN and infinity come last
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  top = max(top, quad_xor<1>(top));
  top = max(top, quad_xor<2>(top));
  const bool finite = top < 0x7f800000u;
  const uint32_t byte = finite ? (uint32_t)max((int)(top >> 23) - 2, 0) : 255u;
  *(uint32_t*)(codes + (r * K + c) / 2) = finite ? codes_of(v, scale_of(byte)) : 0u;
  if (c % 32 == 0) scales[r * sld + c / 32] = (uint8_t)byte;
}

hipError_t launch_quantize_mxfp4(int dtype, int form, const void* x, int64_t src_rows,
                                 const int32_t* row_index, int64_t rows, int K, void* rows_out,
                                 uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int sld = mx_scale_row(K);
  const int64_t chunks = rows * sld * 4;   // of 8 values, over a row and its padding blocks
  if (chunks > (int64_t)1 << 31) return hipErrorInvalidValue;   // 2^27 rows of 32 are 2^31
  const unsigned blocks = (unsigned)((chunks + 255) / 256);
  const Divider per_row = divider((uint32_t)sld * 4);
#define GO(D, F)                                                                               \
  hipLaunchKernelGGL((k_quantize<D, F>), dim3(blocks), dim3(256), 0, stream, (const char*)x,   \
                     src_rows, row_index, (uint32_t)chunks, per_row, K, (char*)rows_out, codes, \
                     scales, sld)
#define BY_FORM(D)                                      \
  do {                                                  \
    if (form == kQuantPlain) GO(D, kQuantPlain);        \
    else if (form == kQuantGather) GO(D, kQuantGather); \
    else GO(D, kQuantSiluMul);                          \
  } while (0)
  if (dtype == 1) BY_FORM(BF16); else BY_FORM(F32);
#undef BY_FORM
#undef GO
  return hipGetLastError();
}

// Two chunks of 8 values a thread, both asked for before either is stored.
template <typename D>
__global__ __launch_bounds__(256) void k_dequantize(const uint8_t* __restrict__ codes,
                                                    const uint8_t* __restrict__ scales,
                                                    uint32_t chunks, Divider per_row, int K,
                                                    char* __restrict__ out, int sld) {
  uint32_t q[2] = {0, 0}, byte[2] = {0, 0};
  const uint32_t first = blockIdx.x * 512 + threadIdx.x;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t i = first + u * 256;
    if (i >= chunks) break;
    const uint32_t row = divide(i, per_row);
    q[u] = *(const uint32_t*)(codes + (int64_t)i * 4);
    byte[u] = scales[(int64_t)row * sld + (i - row * per_row.d) / 4];
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t i = first + u * 256;
    if (i >= chunks) break;
    const float scale = scale_of(byte[u]);
    float v[8];
    // a code by the scale 1 is exact; the product rounds where the type must
#define PAIR(J)                                                                \
  {                                                                            \
    const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.0f, J);   \
    v[2 * J] = p.x * scale;                                                    \
    v[2 * J + 1] = p.y * scale;                                                \
  }
    PAIR(0) PAIR(1) PAIR(2) PAIR(3)
#undef PAIR
    store8<D>(out + (int64_t)i * 8 * D::kBytes, v);
  }
}

hipError_t launch_dequantize_mxfp4(int dtype, const uint8_t* codes, const uint8_t* scales,
                                   int64_t rows, int K, void* out, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int64_t chunks = rows * (K / 8);
  if (chunks > 0x7fffffff) return hipErrorInvalidValue;
  const unsigned blocks = (unsigned)((chunks + 511) / 512);
  const Divider per_row = divider((uint32_t)K / 8);
#define GO(D)                                                                                   \
  hipLaunchKernelGGL(k_dequantize<D>, dim3(blocks), dim3(256), 0, stream, codes, scales,        \
                     (uint32_t)chunks, per_row, K, (char*)out, mx_scale_row(K))
  if (dtype == 1) GO(BF16); else GO(F32);
#undef GO
  return hipGetLastError();
}

}  // namespace lora
