// C ABI of the dense layer's operators: argument validation on the host and
// kernel launches on the caller's stream, by the same rules as lora_api.cpp
// (nothing allocated, nothing synchronised, device data never read here).
#include "lora_mi355x.h"

#include <hip/hip_runtime.h>

#include "dense.h"
#include "linear_choice.h"

namespace {

constexpr int64_t kMaxI32 = 0x7fffffff;
constexpr int64_t kMaxWidth = 1 << 20;
constexpr int64_t k2GiB = (int64_t)1 << 31;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
bool dtype_ok(int dtype) { return dtype == LORA_F32 || dtype == LORA_BF16; }
lora_status hip_status(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_ERR_HIP; }

lora_status check_rows(int64_t rows, int64_t K, int64_t multiple) {
  if (rows < 0 || rows > kMaxI32 || K < 1) return LORA_ERR_INVALID_ARG;
  if (K > kMaxWidth) return LORA_ERR_UNSUPPORTED;
  if (K % multiple != 0) return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}

// e into a; out is the number of W's rows.
lora_status take_epilogue(const lora_epilogue* e, int64_t out, int64_t row_bytes, bool gated,
                          lora::LinearArgs* a) {
  a->bias = a->residual = nullptr;
  a->h = nullptr;
  a->order = nullptr;
  a->act = lora::kActNone;
  a->bias_f32 = 0;
  a->slices = 0;
  if (!e) return LORA_OK;
  if (e->activation < LORA_ACT_NONE || e->activation > LORA_ACT_SILU) return LORA_ERR_INVALID_ARG;
  a->act = e->activation;
  if (e->bias) {
    if (!dtype_ok(e->bias_dtype)) return LORA_ERR_UNSUPPORTED;
    if (!aligned(e->bias, e->bias_dtype == LORA_F32 ? 4 : 2)) return LORA_ERR_ALIGNMENT;
    a->bias = e->bias;
    a->bias_f32 = e->bias_dtype == LORA_F32;
  }
  if (e->residual) {
    if (gated) return LORA_ERR_INVALID_ARG;
    if (!aligned16(e->residual)) return LORA_ERR_ALIGNMENT;
    a->residual = e->residual;
  }
  if (!e->h) return LORA_OK;
  if (e->slots < 1 || e->slots > 8192 || e->R < 1 || e->R > 256 || e->num_slices < 1 ||
      e->num_slices > 8 || e->num_slices * e->R > 1024)
    return LORA_ERR_UNSUPPORTED;
  if (!e->b || !e->token_order || !e->slot_indptr || !e->ranks || !e->scalings || !e->out_slices)
    return LORA_ERR_INVALID_ARG;
  int64_t sum = 0;
  for (int i = 0; i < e->num_slices; ++i) {
    const int64_t w = e->out_slices[i];
    if (w < 1 || w > out - sum) return LORA_ERR_INVALID_ARG;
    if (w % 8 != 0) return LORA_ERR_ALIGNMENT;
    a->off[i] = (int)sum;
    sum += w;
  }
  if (sum != out) return LORA_ERR_INVALID_ARG;
  for (int i = e->num_slices; i < 9; ++i) a->off[i] = (int)sum;
  if (e->R % 8 != 0 || !aligned16(e->h) || !aligned16(e->b)) return LORA_ERR_ALIGNMENT;
  // x and h are reached by 32-bit offsets; a slot's b holds 2^30 bytes at most
  if (a->T * row_bytes >= k2GiB || (int64_t)a->T * e->num_slices * e->R * 4 >= k2GiB)
    return LORA_ERR_UNSUPPORTED;
  a->h = e->h;
  a->b = e->b;
  a->slots = e->slots;
  a->R = e->R;
  a->slices = e->num_slices;
  a->order = e->token_order;
  a->indptr = e->slot_indptr;
  a->ranks = e->ranks;
  a->scalings = e->scalings;
  return LORA_OK;
}

lora_status linear_impl(int operands, bool gated, const void* x, const uint8_t* x_scales, int64_t T,
                        const void* w, const uint8_t* w_scales, int64_t N, int64_t K,
                        const lora_epilogue* e, int dtype, void* y, uint8_t* codes,
                        uint8_t* scales, void* stream) {
  if (operands != LORA_OPERANDS_BF16 && operands != LORA_OPERANDS_MXFP8) return LORA_ERR_UNSUPPORTED;
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  const bool mx = operands == LORA_OPERANDS_MXFP8;
  const lora_status st = check_rows(T, K, mx ? 32 : 8);
  if (st != LORA_OK) return st;
  if (N < 1) return LORA_ERR_INVALID_ARG;
  if (N > kMaxWidth) return LORA_ERR_UNSUPPORTED;
  const int64_t out = gated ? 2 * N : N;
  if (mx && gated && out * lora::mx8_scale_row(K) >= k2GiB) return LORA_ERR_UNSUPPORTED;
  if ((codes == nullptr) != (scales == nullptr)) return LORA_ERR_INVALID_ARG;
  if (codes && N % 32 != 0) return LORA_ERR_ALIGNMENT;
  lora::LinearArgs a = {};
  a.T = (int)T;
  a.N = (int)N;
  a.K = (int)K;
  const lora_status se = take_epilogue(e, out, K * (mx ? 1 : 2), gated, &a);
  if (se != LORA_OK) return se;
  if (T == 0) return LORA_OK;
  if (!x || !w || !y || (mx && (!x_scales || !w_scales))) return LORA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(x_scales) ||
      !aligned16(w_scales) || !aligned16(codes) || !aligned16(scales))
    return LORA_ERR_ALIGNMENT;
  a.x = (const uint8_t*)x;
  a.xs = x_scales;
  a.w = (const uint8_t*)w;
  a.ws = w_scales;
  a.y = y;
  a.y_f32 = dtype == LORA_F32;
  a.codes = codes;
  a.scales = scales;
  const hipStream_t s = (hipStream_t)stream;
  if (mx) return hip_status(gated ? lora::launch_linear_mx8_gated(a, s) : lora::launch_linear_mx8(a, s));
  return hip_status(gated ? lora::launch_linear_bf16_gated(a, s) : lora::launch_linear_bf16(a, s));
}

}  // namespace

extern "C" {

lora_status lora_add_rms_norm(int dtype, const void* x, const void* residual, const void* weight,
                              int64_t T, int64_t width, float eps, float weight_offset, void* rows,
                              void* residual_out, uint8_t* codes, uint8_t* scales, void* stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  if ((codes == nullptr) != (scales == nullptr)) return LORA_ERR_INVALID_ARG;
  const lora_status st = check_rows(T, width, codes ? 32 : 8);
  if (st != LORA_OK) return st;
  if (!(eps >= 0.0f)) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!x || !weight || !rows || (residual == nullptr) != (residual_out == nullptr))
    return LORA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(rows) ||
      !aligned16(residual_out) || !aligned16(codes) || !aligned16(scales))
    return LORA_ERR_ALIGNMENT;
  lora::NormArgs a;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.rows = rows;
  a.residual_out = residual_out;
  a.codes = codes;
  a.scales = scales;
  a.T = (int)T;
  a.H = (int)width;
  a.eps = eps;
  a.offset = weight_offset;
  return hip_status(lora::launch_add_rms_norm(dtype, a, (hipStream_t)stream));
}

int64_t lora_mxfp8_scale_row_bytes(int64_t K) {
  return check_rows(0, K, 32) == LORA_OK ? lora::mx8_scale_row(K) : 0;
}

lora_status lora_quantize_mxfp8(int dtype, const void* x, int64_t rows, int64_t K, uint8_t* codes,
                                uint8_t* scales, void* stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  const lora_status st = check_rows(rows, K, 32);
  if (st != LORA_OK) return st;
  if (rows * lora::mx8_scale_row(K) * 4 > kMaxI32) return LORA_ERR_UNSUPPORTED;
  if (rows == 0) return LORA_OK;
  if (!x || !codes || !scales) return LORA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return LORA_ERR_ALIGNMENT;
  return hip_status(lora::launch_quantize_mxfp8(dtype, x, rows, (int)K, codes, scales, (hipStream_t)stream));
}

lora_status lora_dequantize_mxfp8(int dtype, const uint8_t* codes, const uint8_t* scales,
                                  int64_t rows, int64_t K, void* out, void* stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  const lora_status st = check_rows(rows, K, 32);
  if (st != LORA_OK) return st;
  if (rows * lora::mx8_scale_row(K) * 4 > kMaxI32) return LORA_ERR_UNSUPPORTED;
  if (rows == 0) return LORA_OK;
  if (!codes || !scales || !out) return LORA_ERR_INVALID_ARG;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out)) return LORA_ERR_ALIGNMENT;
  return hip_status(lora::launch_dequantize_mxfp8(dtype, codes, scales, rows, (int)K, out, (hipStream_t)stream));
}

lora_status lora_epilogue_linear(int operands, const void* x, const uint8_t* x_scales, int64_t T,
                                 const void* w, const uint8_t* w_scales, int64_t N, int64_t K,
                                 const lora_epilogue* e, int dtype, void* y, void* stream) {
  return linear_impl(operands, false, x, x_scales, T, w, w_scales, N, K, e, dtype, y, nullptr,
                     nullptr, stream);
}

lora_status lora_gated_linear(int operands, const void* x, const uint8_t* x_scales, int64_t T,
                              const void* w, const uint8_t* w_scales, int64_t N, int64_t K,
                              const lora_epilogue* e, void* rows, uint8_t* codes, uint8_t* scales,
                              void* stream) {
  return linear_impl(operands, true, x, x_scales, T, w, w_scales, N, K, e, LORA_BF16, rows, codes,
                     scales, stream);
}

// Not part of the C ABI: the kernel of a product on `units` compute units, as
// rows, cols and each of LinearChoice, for tests that have to reach all of them.
void lora_test_linear_choice(int mx, int gated, int y_f32, int residual, int T, int N, int K, int units,
                             int32_t* choice) {
  lora::LinearArgs a = {};
  a.T = T;
  a.N = N;
  a.K = K;
  a.y_f32 = y_f32;
  a.residual = residual ? choice : nullptr;   // whether there is one counts
  const lora::LinearChoice c = mx ? (gated ? lora::choose_linear<true, true>(a, units)
                                           : lora::choose_linear<true, false>(a, units))
                                  : (gated ? lora::choose_linear<false, true>(a, units)
                                           : lora::choose_linear<false, false>(a, units));
  choice[0] = c.rows;
  choice[1] = c.cols;
  choice[2] = c.each;
}

}  // extern "C"
