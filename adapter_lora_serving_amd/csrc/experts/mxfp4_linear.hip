// Products over MXFP4 operands: y = x @ W^T for one weight, or per row the
// weight of the expert that the row belongs to.
//
// Page "mstar.model.components.linear", FusedColumnLinear (W [out, in], the
// shards stacked along the output dimension), and page
// "spark_model/lora/expert_apply.rs" (the experts' products on rows sorted
// by expert, before the experts' LoRA is added to them).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 32 codes and a scale byte of each
// operand per lane: lane (m = lane & 15, g = lane >> 4) supplies row m, block
// g of 32 of a K step of 128, and receives D[4g + i][m] in element i. The W
// rows are operand A and the x rows operand B, so a lane ends with 4
// consecutive columns of one row of y. Products of two 4-bit values and the
// powers of two are exact; the sums are fp32, y is rounded once.
#include "lora_common.h"
#include "experts.h"

namespace lora {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma_mx(u32x4 a, u32x4 b, f32x4 c, int sa, int sb) {
  const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, sa, 0, sb);
}

// Segment s of the rows: 0 is the rows before the first expert, 1 .. E the
// experts, E + 1 the rows after the last. Clamped, so malformed offsets give
// wrong values but no access outside the buffers.
__device__ __forceinline__ void segment_rows(const int32_t* __restrict__ offs, int s, int E,
                                             int rows, int& beg, int& n) {
  const int b = s == 0 ? 0 : min(max(offs[s - 1], 0), rows);
  const int e = s == E + 1 ? rows : min(max(offs[s], b), rows);
  beg = b;
  n = max(e - b, 0);
}

}  // namespace

// 64 x 64 tile of y, 4 waves of 32 x 32, operands straight from memory.
template <typename D>
__global__ __launch_bounds__(256) void k_mx_simple(MxArgs a, int sld) {
  __shared__ int scratch[24];
  const int lane = lane_id();
  const int w = wave_id();
  const int m = lane & 15, g = lane >> 4;
  int beg = 0, n = a.rows, e = 0, tile = blockIdx.y;
  bool zero = false;
  if (a.offsets) {
    const SlotItem it = locate_item(
        (int)blockIdx.y, a.E + 2,
        [&](int s) {
          int b, c;
          segment_rows(a.offsets, s, a.E, a.rows, b, c);
          return (c + 63) / 64;
        },
        scratch);
    if (it.slot < 0) return;
    segment_rows(a.offsets, it.slot, a.E, a.rows, beg, n);
    e = it.slot - 1;
    zero = e < 0 || e >= a.E;
    if (zero) e = 0;
    tile = it.local;
  }
  const int r0 = tile * 64 + (w & 1) * 32;         // within the segment
  const int c0 = blockIdx.x * 64 + (w >> 1) * 32;
  const int kb = a.K / 32;
  const int64_t rowb = a.K / 2;
  const uint8_t* W = a.w + (int64_t)e * a.N * rowb;
  const uint8_t* WS = a.ws + (int64_t)e * a.N * sld;
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (!zero) {
    for (int b0 = 0; b0 < kb; b0 += 4) {
      const int b = b0 + g;
      u32x4 xo[2], wo[2];
      int xsc[2], wsc[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + i * 16 + m, c = c0 + i * 16 + m;
        xo[i] = wo[i] = u32x4{0u, 0u, 0u, 0u};
        xsc[i] = wsc[i] = 0;
        if (b < kb && r < n) {
          xo[i] = *(const u32x4*)(a.x + (int64_t)(beg + r) * rowb + b * 16);
          xsc[i] = a.xs[(int64_t)(beg + r) * sld + b];
        }
        if (b < kb && c < a.N) {
          wo[i] = *(const u32x4*)(W + (int64_t)c * rowb + b * 16);
          wsc[i] = WS[(int64_t)c * sld + b];
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma_mx(wo[i], xo[j], acc[i][j], wsc[i], xsc[j]);
    }
  }
  // wait states between the last MFMA and the first vector read of its result
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = r0 + j * 16 + m, c = c0 + i * 16 + 4 * g + q;
        if (r < n && c < a.N) {
          const int64_t at = (int64_t)(beg + r) * a.N + c;
          if constexpr (D::kBytes == 2)
            ((uint16_t*)a.y)[at] = (uint16_t)to_bf16_bits(acc[i][j][q]);
          else
            ((float*)a.y)[at] = acc[i][j][q];
        }
      }
}

hipError_t launch_mxfp4_linear(int dtype, const MxArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  const int sld = mx_scale_row(a.K);
  // tiles of a segmented batch: one more per segment for its ragged end
  const int64_t mt = (a.rows + 63) / 64 + (a.offsets ? a.E + 2 : 0);
  const int64_t nt = (a.N + 63) / 64;
  if (mt > 65535 * 4 || nt > 0x7fffffff) return hipErrorInvalidValue;
#define GO(D)                                                                                \
  hipLaunchKernelGGL(k_mx_simple<D>, dim3((unsigned)nt, (unsigned)mt), dim3(256), 0, stream, a, sld)
  if (dtype == 1) GO(BF16); else GO(F32);
#undef GO
  return hipGetLastError();
}

}  // namespace lora
