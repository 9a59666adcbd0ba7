// The Python binding of the dense layer's operators, compiled for the reason
// that the routed-expert one is: a decode step's operators take less time on
// the GPU than a call by way of ctypes on the host.
//
// Each function takes its arguments by position, as dense.py gives them.
#include "python/binding.h"

#include <vector>

namespace {

bool is_e4m3(at::ScalarType t) { return t == at::kFloat8_e4m3fn || t == at::kByte; }

// An operand: rows of K values, bf16 or an MXFP8 pair.
struct Operand {
  bool mx = false;
  at::Tensor codes, scales;
  int64_t rows = 0, K = 0;
};

void take_pair(Call& c, PyObject* pair, const char* name, Operand& o) {
  o.mx = true;
  o.codes = c.tensor(PyTuple_GET_ITEM(pair, 0), name);
  o.scales = c.tensor(PyTuple_GET_ITEM(pair, 1), name);
  const int64_t d = o.codes.dim();
  bool ok = d >= 1 && o.scales.dim() == d && is_e4m3(o.codes.scalar_type()) &&
            o.scales.scalar_type() == at::kByte;
  if (ok) {
    o.K = o.codes.size(d - 1);
    o.rows = 1;
    for (int64_t i = 0; i + 1 < d; ++i) {
      ok = ok && o.scales.size(i) == o.codes.size(i);
      o.rows *= o.codes.size(i);
    }
    const int64_t ld = lora_mxfp8_scale_row_bytes(o.K);
    ok = ok && ld > 0 && o.scales.size(d - 1) == ld;
  }
  if (!ok)
    refuse("%s: codes must be float8_e4m3fn [..., K], K a multiple of 32, and scales uint8 "
           "[..., K / 32 rounded up to a multiple of 16]", name);
}

bool is_pair(PyObject* o) { return PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2; }

Operand operand(Call& c, PyObject* o, const char* name) {
  Operand r;
  if (is_pair(o)) {
    take_pair(c, o, name, r);
  } else {
    r.codes = c.tensor(o, name);
    if (r.codes.scalar_type() != at::kBFloat16 || r.codes.dim() < 1)
      refuse("%s must be bf16 [..., K] or an MXFP8 pair (codes, scales)", name);
    r.K = r.codes.size(-1);
    r.rows = r.K > 0 ? r.codes.numel() / r.K : 0;
  }
  if (r.codes.dim() != 2) refuse("%s must have two dimensions", name);
  return r;
}

// The error of an argument of another kind goes, any other stays and is raised.
void not_that() {
  if (!PyErr_ExceptionMatches(PyExc_TypeError) && !PyErr_ExceptionMatches(PyExc_ValueError) &&
      !PyErr_ExceptionMatches(PyExc_OverflowError))
    throw python_error();
  PyErr_Clear();
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    not_that();
    refuse("%s must be a number", name);
  }
  return v;
}

// The epilogue's arguments, and what keeps their tensors alive over the call.
struct Epilogue {
  lora_epilogue e = {};
  Opt bias, residual, h, b, order, indptr, ranks, scalings;
  std::vector<int64_t> slices;
};

// (h, b, addressing, ranks, scalings, out_slices)
void take_delta(Call& c, PyObject* d, int64_t T, int64_t out, Epilogue& p) {
  if (!PyTuple_Check(d) || PyTuple_GET_SIZE(d) != 6)
    refuse("delta must be a Delta (h, b, addressing, ranks, scalings, out_slices)");
  p.h = c.tensor(PyTuple_GET_ITEM(d, 0), "delta.h");
  p.b = c.tensor(PyTuple_GET_ITEM(d, 1), "delta.b");
  PyObject* addr = PyTuple_GET_ITEM(d, 2);
  if (!is_pair(addr)) refuse("delta.addressing must be an Addressing");
  p.order = c.int32(PyTuple_GET_ITEM(addr, 0), "token_order");
  p.indptr = c.int32(PyTuple_GET_ITEM(addr, 1), "slot_indptr");
  p.ranks = c.int32(PyTuple_GET_ITEM(d, 3), "delta.ranks");
  p.scalings = c.tensor(PyTuple_GET_ITEM(d, 4), "delta.scalings");
  PyObject* seq = PySequence_Fast(PyTuple_GET_ITEM(d, 5), "");
  if (!seq) {
    not_that();
    refuse("delta.out_slices must be a sequence");
  }
  bool whole = true;
  for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq) && whole; ++i) {
    const int64_t w = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
    if (w == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      whole = false;
    }
    p.slices.push_back(w);
  }
  Py_DECREF(seq);
  if (!whole) refuse("delta.out_slices must be integers");
  const int64_t S = (int64_t)p.slices.size();
  if (p.b->dim() != 3 || p.b->size(1) != out || p.b->scalar_type() != at::kBFloat16)
    refuse("delta.b must be bf16 [slots, %lld, R]", (long long)out);
  const int64_t slots = p.b->size(0), R = p.b->size(2);
  if (S < 1 || S > 8 || slots > INT32_MAX || R > INT32_MAX) refuse("delta: too many slices, slots or ranks");
  given(*p.h, T, S * R, at::kFloat, "delta.h");
  if (p.order->numel() != T || p.indptr->numel() != slots + 1)
    refuse("delta.addressing must be [T] and [slots + 1]");
  if (p.ranks->numel() != slots || p.scalings->numel() != slots ||
      p.scalings->scalar_type() != at::kFloat)
    refuse("delta.ranks and delta.scalings must be [slots], scalings float32");
  p.e.h = as<const float>(p.h);
  p.e.b = ptr(p.b);
  p.e.slots = (int32_t)slots;
  p.e.R = (int32_t)R;
  p.e.token_order = as<const int32_t>(p.order);
  p.e.slot_indptr = as<const int32_t>(p.indptr);
  p.e.ranks = as<const int32_t>(p.ranks);
  p.e.scalings = as<const float>(p.scalings);
  p.e.out_slices = p.slices.data();
  p.e.num_slices = (int32_t)S;
}

void take_bias(Call& c, PyObject* o, int64_t out, Epilogue& p) {
  p.bias = c.optional(o, "bias");
  if (!p.bias) return;
  if (p.bias->dim() != 1 || p.bias->numel() != out) refuse("bias must be [%lld]", (long long)out);
  p.e.bias_dtype = dtype_code(p.bias->scalar_type());
  p.e.bias = ptr(p.bias);
}

struct Product {
  Operand x, w;
  int operands = 0;
};
Product product(Call& c, PyObject* x, PyObject* w, const char* what) {
  Product p;
  p.x = operand(c, x, "x");
  p.w = operand(c, w, "w");
  if (p.x.mx != p.w.mx) refuse("%s: x and w must both be bf16 or both MXFP8", what);
  if (p.x.K != p.w.K) refuse("%s: shape mismatch between x and w", what);
  p.operands = p.x.mx ? LORA_OPERANDS_MXFP8 : LORA_OPERANDS_BF16;
  return p;
}
const uint8_t* scales_of(const Operand& o) { return o.mx ? as<const uint8_t>(o.scales) : nullptr; }

// (x, w, bias, activation, residual, delta, dtype, y) -> (y,)
PyObject* linear(PyObject* const* a) {
  Call c;
  const Product p = product(c, a[0], a[1], "epilogue_linear");
  const int64_t T = p.x.rows, N = p.w.rows;
  Epilogue e;
  take_bias(c, a[2], N, e);
  e.e.activation = integer32(a[3], "activation");
  e.residual = c.optional(a[4], "residual");
  if (a[5] != Py_None) take_delta(c, a[5], T, N, e);
  const Opt y_in = c.optional(a[7], "y");
  const at::ScalarType st = dtype_arg(a[6], y_in ? y_in->scalar_type() : at::kBFloat16);
  const int dt = dtype_code(st);
  if (y_in) given(*y_in, T, N, st, "y");
  if (e.residual) given(*e.residual, T, N, st, "residual");
  e.e.residual = ptr(e.residual);
  const c10::DeviceGuard guard(p.x.codes.device());
  const at::Tensor y = y_in ? *y_in : c.make({T, N}, st);
  check(lora_epilogue_linear(p.operands, ptr(p.x.codes), scales_of(p.x), T, ptr(p.w.codes),
                             scales_of(p.w), N, p.x.K, &e.e, dt, ptr(y), c.stream()),
        "lora_epilogue_linear");
  return pack({&y});
}

// (x, w, bias, activation, delta, held, y) -> (rows, codes or None, scales or None)
PyObject* gated(PyObject* const* a) {
  Call c;
  const Product p = product(c, a[0], a[1], "gated_linear");
  if (p.w.rows % 2) refuse("gated_linear: w must hold as many gates as ups");
  const int64_t T = p.x.rows, N = p.w.rows / 2;
  Epilogue e;
  take_bias(c, a[2], 2 * N, e);
  e.e.activation = integer32(a[3], "activation");
  if (a[4] != Py_None) take_delta(c, a[4], T, 2 * N, e);
  const bool held = a[5] == Py_True;
  const Opt y_in = c.optional(a[6], "y");
  if (y_in) given(*y_in, T, N, at::kBFloat16, "y");
  const int64_t ld = held ? lora_mxfp8_scale_row_bytes(N) : 0;
  if (held && ld == 0) refuse("gated_linear: rows in MXFP8 must be a multiple of 32 wide, at most 2^20");
  const c10::DeviceGuard guard(p.x.codes.device());
  const at::Tensor y = y_in ? *y_in : c.make({T, N}, at::kBFloat16);
  Opt codes, scales;
  if (held) {
    codes = c.make({T, N}, at::kFloat8_e4m3fn);
    scales = c.make({T, ld}, at::kByte);
  }
  check(lora_gated_linear(p.operands, ptr(p.x.codes), scales_of(p.x), T, ptr(p.w.codes),
                          scales_of(p.w), N, p.x.K, &e.e, ptr(y), as<uint8_t>(codes),
                          as<uint8_t>(scales), c.stream()),
        "lora_gated_linear");
  return pack({&y, codes ? &*codes : nullptr, scales ? &*scales : nullptr});
}

// (x, weight, residual, eps, offset, held, residual_out) -> (rows, residual_out, codes, scales)
PyObject* norm(PyObject* const* a) {
  const double eps = number(a[3], "eps"), offset = number(a[4], "weight_offset");
  Call c;
  const at::Tensor x = c.tensor(a[0], "x"), weight = c.tensor(a[1], "weight");
  if (x.dim() != 2) refuse("x must be [T, width]");
  const int64_t T = x.size(0), H = x.size(1);
  const int dt = dtype_code(x.scalar_type());
  if (weight.dim() != 1 || weight.numel() != H || weight.scalar_type() != x.scalar_type())
    refuse("weight must be [width] of x's type");
  const Opt residual = c.optional(a[2], "residual"), out_in = c.optional(a[6], "residual_out");
  if (residual) given(*residual, T, H, x.scalar_type(), "residual");
  if (out_in && !residual) refuse("residual_out goes with a residual");
  if (out_in) given(*out_in, T, H, x.scalar_type(), "residual_out");
  const bool held = a[5] == Py_True;
  const int64_t ld = held ? lora_mxfp8_scale_row_bytes(H) : 0;
  if (held && ld == 0) refuse("rows in MXFP8 must be a multiple of 32 wide, at most 2^20");
  const c10::DeviceGuard guard(x.device());
  const at::Tensor rows = c.make({T, H}, x.scalar_type());
  Opt res_out, codes, scales;
  if (residual) res_out = out_in ? *out_in : c.make({T, H}, x.scalar_type());
  if (held) {
    codes = c.make({T, H}, at::kFloat8_e4m3fn);
    scales = c.make({T, ld}, at::kByte);
  }
  check(lora_add_rms_norm(dt, ptr(x), ptr(residual), ptr(weight), T, H, (float)eps, (float)offset,
                          ptr(rows), ptr(res_out), as<uint8_t>(codes), as<uint8_t>(scales),
                          c.stream()),
        "lora_add_rms_norm");
  return pack({&rows, res_out ? &*res_out : nullptr, codes ? &*codes : nullptr,
               scales ? &*scales : nullptr});
}

// (x,) -> (codes, scales), of x's leading dimensions
PyObject* quantize(PyObject* const* a) {
  Call c;
  const at::Tensor x = c.tensor(a[0], "x");
  if (x.dim() < 1) refuse("x must be [..., K]");
  const int dt = dtype_code(x.scalar_type());
  const int64_t K = x.size(-1), ld = lora_mxfp8_scale_row_bytes(K);
  if (ld == 0) refuse("K must be a multiple of 32, at most 2^20");
  const int64_t n = x.numel() / K;
  const c10::DeviceGuard guard(x.device());
  std::vector<int64_t> shape = x.sizes().vec();
  const at::Tensor codes = c.make(shape, at::kFloat8_e4m3fn);
  shape.back() = ld;
  const at::Tensor scales = c.make(shape, at::kByte);
  check(lora_quantize_mxfp8(dt, ptr(x), n, K, as<uint8_t>(codes), as<uint8_t>(scales), c.stream()),
        "lora_quantize_mxfp8");
  return pack({&codes, &scales});
}

// (pair, dtype or None) -> (values,)
PyObject* dequantize(PyObject* const* a) {
  Call c;
  if (!is_pair(a[0])) refuse("dequantize_mxfp8: an MXFP8 pair (codes, scales)");
  Operand q;
  take_pair(c, a[0], "dequantize_mxfp8", q);
  const at::ScalarType st = dtype_arg(a[1], at::kBFloat16);
  const int dt = dtype_code(st);
  const c10::DeviceGuard guard(q.codes.device());
  const at::Tensor out = c.make(q.codes.sizes(), st);
  check(lora_dequantize_mxfp8(dt, as<const uint8_t>(q.codes), as<const uint8_t>(q.scales), q.rows,
                              q.K, ptr(out), c.stream()),
        "lora_dequantize_mxfp8");
  return pack({&out});
}

PyMethodDef methods[] = {ENTRY(setup, 2),    ENTRY(linear, 8),     ENTRY(gated, 7), ENTRY(norm, 7),
                         ENTRY(quantize, 1), ENTRY(dequantize, 2), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__dense(void) { return PyModule_Create(&module); }
