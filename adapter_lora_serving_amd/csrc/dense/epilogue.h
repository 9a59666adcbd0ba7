// What the products of the dense layer share: activations, matrix
// instructions over both operand forms, the LoRA delta on their accumulators.
#pragma once

#include "dense.h"
#include "mx8.h"

namespace lora {

typedef int i32x8 __attribute__((ext_vector_type(8)));
// 16 bytes from any element on: rows of y start where they start
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

constexpr float kLog2e = 1.44269504088896340736f;

// Activations in fp32. silu and the tanh form of gelu are z times a logistic
// function of u = z or 2 sqrt(2 / pi) (z + 0.044715 z^3), one v_exp_f32 and one
// v_rcp_f32 (1 ulp each). The exponent's argument is off by at most 2^-23 |u|
// (silu: a constant and a product) or 2^-21 |u| (eight roundings on the way of
// the cube), so the relative errors are at most (|u| + 4) 2^-23 and (4 |u| + 4)
// 2^-23, where the function is not yet flat.
__device__ __forceinline__ float logistic_times(float z, float t) {   // z / (1 + 2^t)
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}
// z Phi(z), Phi the normal distribution function. Phi(-a) = exp(-a^2 / 2) t P(t)
// for a >= 0 with t = 1 / (1 + 0.275 a): P is the polynomial of degree 8 whose
// largest relative error over all a is least (6e-8), found by weighted least
// squares on the scaled complementary error function. a^2 / 2 and its product
// with log2 e keep what their roundings drop, or the tail would be off by a^2 2^-24.
// So the relative error is the same on both sides: at most 2^-19 by adding up
// the roundings, 4.8e-7 measured over |z| < 13.
__device__ __forceinline__ float gelu_erf(float z) {
  const float a = fminf(fabsf(z), 16.0f);   // where Phi(-a) is 0 in fp32; no infinity from here on
  const float t = __builtin_amdgcn_rcpf(fmaf(0.275f, a, 1.0f));
  float p = fmaf(2.716985390e-2f, t, -1.106834245e-1f);
  p = fmaf(p, t, 1.301848217e-1f);
  p = fmaf(p, t, -3.517562190e-2f);
  p = fmaf(p, t, 8.801499072e-2f);
  p = fmaf(p, t, 7.893343728e-2f);
  p = fmaf(p, t, 1.021909300e-1f);
  p = fmaf(p, t, 1.096543131e-1f);
  p = fmaf(p, t, 1.097106876e-1f);
  constexpr double kHalf = 0.72134752044448170368;   // log2 e / 2
  constexpr float kHi = (float)kHalf, kLo = (float)(kHalf - (double)kHi);
  const float s = a * a, ds = fmaf(a, a, -s);
  const float u = s * kHi, du = fmaf(s, kLo, fmaf(ds, kHi, fmaf(s, kHi, -u)));
  float e = __builtin_amdgcn_exp2f(-u);
  e = fmaf(e, du * -0.69314718055994530942f, e);
  const float q = p * t * e;
  return z * (z > 0.0f ? 1.0f - q : q);
}
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;   // a NaN stays one
    case kActGelu: return gelu_erf(z);
    case kActGeluTanh: {
      constexpr float c = -2.0f * 0.79788456080286535588f * kLog2e;
      return logistic_times(z, z * fmaf(c * 0.044715f, z * z, c));
    }
    case kActSilu: return logistic_times(z, z * -kLog2e);
    default: return z;
  }
}

template <int N>
__device__ __forceinline__ void activate_run(int act, float* v) {
  switch (act) {   // the same for every lane
    case kActNone: break;
    case kActRelu: _Pragma("unroll") for (int e = 0; e < N; ++e) v[e] = activate(kActRelu, v[e]); break;
    case kActGelu: _Pragma("unroll") for (int e = 0; e < N; ++e) v[e] = activate(kActGelu, v[e]); break;
    case kActGeluTanh: _Pragma("unroll") for (int e = 0; e < N; ++e) v[e] = activate(kActGeluTanh, v[e]); break;
    default: _Pragma("unroll") for (int e = 0; e < N; ++e) v[e] = activate(kActSilu, v[e]); break;
  }
}

// The larger of v in lanes L and L ^ 32, for both.
__device__ __forceinline__ uint32_t max_of_halves(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)r[0], (uint32_t)r[1]);
}

// Two values in bf16 by one v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// ---- 8 columns of one row of y --------------------------------------------

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}
__device__ __forceinline__ float value_at(const void* p, bool f32, int64_t i) {
  return f32 ? ((const float*)p)[i] : bf16_at(p, i);
}

// 8 values in flight: 32 bytes, or 16 of bf16 in the first half
struct Raw8 {
  u32x4 a, b;
  __device__ __forceinline__ void load(const void* p, bool f32, int64_t i) {
    if (f32) {
      a = *(const u32x4_any*)((const float*)p + i);
      b = *(const u32x4_any*)((const float*)p + i + 4);
    } else {
      a = *(const u32x4_any*)((const uint16_t*)p + i);
    }
  }
  __device__ __forceinline__ void add_to(bool f32, float* v) const {
    if (f32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] += __uint_as_float(a[k]);
        v[4 + k] += __uint_as_float(b[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] += bf16lo(a[k]);
        v[2 * k + 1] += bf16hi(a[k]);
      }
    }
  }
};

// What a lane's columns meet, asked for ahead of time where all 8 exist.
template <bool GATED>
struct Ahead {
  Raw8 bias, ubias, res[2];
  __device__ __forceinline__ void load_bias(const LinearArgs& a, int c) {
    if (a.bias && c + 8 <= a.N) {
      bias.load(a.bias, a.bias_f32, c);
      if constexpr (GATED) ubias.load(a.bias, a.bias_f32, a.N + c);
    }
  }
  __device__ __forceinline__ void load_residual(const LinearArgs& a, int k, int64_t at, int c) {
    if (c + 8 <= a.N) res[k].load(a.residual, a.y_f32, at);
  }
};

// Columns [c, c + 8) of row t of y from their products (gated: and the ups'),
// the delta in them. Of a gated product with codes four lanes side by side
// hold a block of 32, whose columns exist together.
template <bool GATED>
__device__ __forceinline__ void finish(const LinearArgs& a, const Ahead<GATED>& n, int k, bool live,
                                       int64_t t, int c, float* v, float* up) {
  const int64_t at = t * a.N + c;
  if (c + 8 > a.N) {   // the last columns of a ragged row, one by one
    for (int i = 0; i < a.N - c; ++i) {
      float z = v[0], z2 = GATED ? up[0] : 0.0f;
#pragma unroll
      for (int q = 1; q < 8; ++q) {
        z = i == q ? v[q] : z;
        if constexpr (GATED) z2 = i == q ? up[q] : z2;
      }
      if (a.bias) {
        z += value_at(a.bias, a.bias_f32, c + i);
        if constexpr (GATED) z2 += value_at(a.bias, a.bias_f32, a.N + c + i);
      }
      z = activate(a.act, z);
      if constexpr (GATED) z *= z2;
      if (!live) continue;
      if (!GATED && a.residual) z += value_at(a.residual, a.y_f32, at + i);
      if (!GATED && a.y_f32)
        ((float*)a.y)[at + i] = z;
      else
        ((uint16_t*)a.y)[at + i] = (uint16_t)to_bf16_bits(z);
    }
    return;
  }
  if (a.bias) {
    n.bias.add_to(a.bias_f32, v);
    if constexpr (GATED) n.ubias.add_to(a.bias_f32, up);
  }
  activate_run<8>(a.act, v);
  if constexpr (GATED) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= up[q];
  } else {
    if (a.residual) n.res[k].add_to(a.y_f32, v);
    if (a.y_f32) {
      if (live) {
        float* dst = (float*)a.y + at;
        *(f32x4_any*)dst = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4_any*)(dst + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
      return;
    }
  }
  const u32x4 o = u32x4{pair_bf16(v[0], v[1]), pair_bf16(v[2], v[3]), pair_bf16(v[4], v[5]),
                        pair_bf16(v[6], v[7])};
  if (live) *(u32x4_any*)((uint16_t*)a.y + at) = o;
  if constexpr (GATED) {
    if (a.codes) {   // MXFP8 of the rounded rows; N is a multiple of 32
      float r[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) { r[2 * q] = bf16lo(o[q]); r[2 * q + 1] = bf16hi(o[q]); }
      uint32_t byte;
      const u32x2 z = mx8_quantize8(r, byte);
      if (live) {
        *(u32x2*)(a.codes + at) = z;
        if (c % 32 == 0) {
          const int ld = mx8_scale_row(a.N), last = a.N / 32;
          uint8_t* sc = a.scales + t * ld;
          sc[c / 32] = (uint8_t)byte;
          if (c / 32 == last - 1)   // the padding of the scale row
            for (int q = last; q < ld; ++q) sc[q] = 0;
        }
      }
    }
  }
}

// D[32x32] += A[32 x 16] . B[32 x 16]^T in bf16: lane (m = lane & 31, h =
// lane >> 5) supplies row m, k in [8 h, 8 h + 8) of both operands and receives
// D[8 (i / 4) + 4 h + i % 4][m] in element i.
__device__ __forceinline__ f32x16 mfma_bf16(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Workgroup barrier that waits for the wave's LDS operations alone.
constexpr int vm_lds_le(int n) { return vmcnt_le(n) & ~(15 << 8); }

// h of a token, scaled, as `TERMS` bf16 parts whose sum it is: the high part
// and what that leaves, so that the delta has h in 16 bits of fraction (2
// terms) or all of its 24 (3 terms). Values that do not fit bf16 show in the
// high part and are not for the matrix unit.
template <int TERMS>
__device__ __forceinline__ void split_bf16(const float* v, u32x4* out) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float x = v[e], y = v[e + 1];
#pragma unroll
    for (int p = 0; p < TERMS; ++p) {
      const uint32_t pair = pair_bf16(x, y);
      out[p][e / 2] = pair;
      if (p + 1 == TERMS) break;
      x -= bf16lo(pair);
      y -= bf16hi(pair);
    }
  }
}

// What the delta's values that do not fit bf16 (lora_common.h) come to for token t
// at position p, added to v: columns [n, n + 8) of W's rows from `first` on.
// Seldom called, so it is short code, not fast code.
__device__ __forceinline__ void add_unfit(const LinearArgs& a, int64_t t, int p, int first, int n,
                                          int64_t out, f32x4* v) {
  const int s = slot_of_position(a.indptr, a.slots, p);
  if (s >= a.slots) return;
  int beg, len;
  segment_of(a.indptr, s, a.T, beg, len);
  if (p < beg || p >= beg + len) return;
  const int r = clamp_rank(a.ranks[s], a.R);
  const float scale = a.scalings[s];
#pragma unroll 1
  for (int q = 0; q < 8 && n + q < a.N; ++q) {
    const int row = first + n + q;
    int si = 0;
    while (si + 1 < a.slices && a.off[si + 1] <= row) ++si;
    const float* h = a.h + (t * a.slices + si) * a.R;
    const uint16_t* b = (const uint16_t*)a.b + (s * out + row) * a.R;
    const float z = unfit_sum(h, b, r, scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i / 4][i % 4] += i == q ? z : 0.0f;
  }
}

// Slot of position p of token_order, found by a wave: the last s with
// indptr[s] <= p, or `slots` for a token without an adapter.
__device__ __forceinline__ int wave_slot_of(const int32_t* __restrict__ indptr, int slots, int p) {
  int n = 0;
  for (int s0 = 0; s0 <= slots; s0 += kWave) {
    const int s = s0 + lane_id();
    n += __popcll(__ballot(s <= slots && indptr[min(s, slots)] <= p));
  }
  return __builtin_amdgcn_readfirstlane(max(n - 1, 0));
}

}  // namespace lora
