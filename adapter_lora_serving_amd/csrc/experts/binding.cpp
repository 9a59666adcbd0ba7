// The Python binding of the routed-expert operators: checks of the tensors,
// outputs from torch's allocator, torch's current stream, and the call of the
// C ABI. Compiled rather than by way of ctypes because a decode step's
// operators take less time on the GPU than such a call on the host: routing
// one token is 8.1 us a call by way of ctypes (3.4 us of it the launch).
//
// Each function takes its arguments by position, as experts.py gives them.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/clamp.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <optional>
#include <string>

#include "lora_mi355x.h"

namespace {

PyObject* g_error = nullptr;   // the package's LoraError
PyObject* g_stream = nullptr;  // torch's current raw stream, by device index

// A LoraError on its way to Python.
struct Refused {};

[[noreturn]] void refuse(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(g_error, fmt, ap);
  va_end(ap);
  throw Refused();
}

void check(lora_status st, const char* what) {
  if (st != LORA_OK) refuse("%s: %s (status %d)", what, lora_status_string(st), (int)st);
}

using Opt = std::optional<at::Tensor>;

// The tensors of a call, all contiguous and on one GPU.
struct Call {
  int dev = -1;

  at::Tensor tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("all tensors must be on the GPU (no CPU fallback)");
    if (!t.is_contiguous()) refuse("tensors must be contiguous (%s)", name);
    const int d = t.device().index();
    if (dev < 0) dev = d;
    if (d != dev) refuse("tensors on different devices");
    return t;
  }
  Opt optional(PyObject* o, const char* name) {
    if (o == Py_None) return std::nullopt;
    return tensor(o, name);
  }
  // Indices as int32. What a wider type holds past int32 becomes int32's end
  // and so stays out of range: cut to 32 bits, 2^32 + 3 would be index 3.
  at::Tensor int32(PyObject* o, const char* name) {
    at::Tensor t = tensor(o, name);
    const at::ScalarType st = t.scalar_type();
    if (st == at::kInt) return t;
    if (st == at::kUInt32 || st == at::kUInt64) t = t.to(at::kLong);
    if (t.scalar_type() == at::kLong) t = at::clamp(t, INT32_MIN, INT32_MAX);
    return t.to(at::kInt);
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType dtype) const {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, (c10::DeviceIndex)dev));
  }
  void* stream() const {
    PyObject* d = PyLong_FromLong(dev);
    PyObject* s = d ? PyObject_CallOneArg(g_stream, d) : nullptr;
    Py_XDECREF(d);
    if (!s) throw python_error();
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw python_error();
    return p;
  }
};

int dtype_code(at::ScalarType t) {
  if (t == at::kBFloat16) return LORA_BF16;
  if (t == at::kFloat) return LORA_F32;
  refuse("unsupported dtype %s (bf16 or fp32)", c10::toString(t));
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s must be an integer", name);
  }
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse("%s is out of range", name);
  return (int32_t)v;
}

// dtype: a torch.dtype, or None for `otherwise`.
at::ScalarType dtype_arg(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) refuse("dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

void given(const at::Tensor& t, int64_t n, int64_t m, at::ScalarType dtype, const char* name) {
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != m || t.scalar_type() != dtype)
    refuse("%s must be %s [%lld, %lld]", name, c10::toString(dtype), (long long)n, (long long)m);
}

void* ptr(const at::Tensor& t) { return t.data_ptr(); }
void* ptr(const Opt& t) { return t ? t->data_ptr() : nullptr; }
template <typename T, typename V>
T* as(const V& t) { return static_cast<T*>(ptr(t)); }

// An MXFP4 pair: rows (all leading dimensions) and K.
struct Held {
  at::Tensor codes, scales;
  int64_t rows = 0, K = 0;
};

Held held(Call& c, PyObject* pair, const char* name) {
  if (!PyTuple_Check(pair) || PyTuple_GET_SIZE(pair) != 2)
    refuse("%s must be an MXFP4 pair (codes, scales)", name);
  Held h;
  h.codes = c.tensor(PyTuple_GET_ITEM(pair, 0), name);
  h.scales = c.tensor(PyTuple_GET_ITEM(pair, 1), name);
  const int64_t d = h.codes.dim();
  bool ok = d >= 1 && h.scales.dim() == d && h.codes.scalar_type() == at::kByte &&
            h.scales.scalar_type() == at::kByte;
  if (ok) {
    h.K = h.codes.size(d - 1) * 2;
    h.rows = 1;
    for (int64_t i = 0; i + 1 < d; ++i) {
      ok = ok && h.scales.size(i) == h.codes.size(i);
      h.rows *= h.codes.size(i);
    }
    ok = ok && h.scales.size(d - 1) == lora_mxfp4_scale_row_bytes(h.K);
  }
  if (!ok)
    refuse("%s: codes must be uint8 [..., K / 2], K a multiple of 32, and scales uint8 "
           "[..., K / 32 rounded up to a multiple of 4]", name);
  return h;
}

PyObject* pack(std::initializer_list<const at::Tensor*> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o = nullptr;
    if (t) {
      o = THPVariable_Wrap(*t);
    } else {
      Py_INCREF(Py_None);
      o = Py_None;
    }
    if (!o) {
      Py_DECREF(out);
      throw python_error();
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// (logits, top_k, scores, bias, groups, top_groups, group_score, renormalize,
//  scaling, ids or None, weights or None) -> (ids, weights)
PyObject* route(PyObject* const* a) {
  Call c;
  const at::Tensor x = c.tensor(a[0], "logits");
  if (x.dim() != 2) refuse("logits must be [T, experts]");
  const int64_t T = x.size(0), E = x.size(1);
  const int32_t k = integer32(a[1], "top_k");
  const Opt bias = c.optional(a[3], "bias");
  if (bias && (bias->scalar_type() != at::kFloat || bias->numel() != E))
    refuse("bias must be float32 [experts]");
  if (k < 1 || E > INT32_MAX) refuse("top_k must be at least 1");
  const int dt = dtype_code(x.scalar_type());
  const Opt ids_in = c.optional(a[9], "ids"), w_in = c.optional(a[10], "weights");
  if (ids_in) given(*ids_in, T, k, at::kInt, "ids");
  if (w_in) given(*w_in, T, k, at::kFloat, "weights");
  const c10::DeviceGuard guard(x.device());
  const at::Tensor ids = ids_in ? *ids_in : c.make({T, k}, at::kInt);
  const at::Tensor w = w_in ? *w_in : c.make({T, k}, at::kFloat);
  const int renormalize = PyObject_IsTrue(a[7]);
  if (renormalize < 0) throw python_error();
  const double scaling = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) throw python_error();
  check(lora_route_experts(dt, ptr(x), T, (int32_t)E, k, integer32(a[2], "scores"),
                           as<const float>(bias), integer32(a[4], "groups"),
                           integer32(a[5], "top_groups"), integer32(a[6], "group_score"),
                           renormalize, (float)scaling, as<int32_t>(ids),
                           as<float>(w), c.stream()),
        "lora_route_experts");
  return pack({&ids, &w});
}

// (ids, num_experts, token_slot or None) -> (row_token, positions, offsets, row_slot or None)
PyObject* rows(PyObject* const* a) {
  Call c;
  const at::Tensor ids = c.int32(a[0], "ids");
  if (ids.dim() != 2) refuse("ids must be [T, top_k]");
  const int64_t T = ids.size(0), k = ids.size(1), n = T * k;
  const int32_t E = integer32(a[1], "num_experts");
  if (E < 1 || k > INT32_MAX) refuse("num_experts must be at least 1");
  Opt slot;
  if (a[2] != Py_None) slot = c.int32(a[2], "token_slot");
  if (slot && slot->numel() != T) refuse("token_slot must be [T]");
  const c10::DeviceGuard guard(ids.device());
  const at::Tensor row_token = c.make({n}, at::kInt), positions = c.make({T, k}, at::kInt),
                   offsets = c.make({(int64_t)E + 1}, at::kInt);
  Opt row_slot, ws;
  if (slot) row_slot = c.make({n}, at::kInt);
  const size_t need = lora_expert_rows_workspace_bytes(T, (int32_t)k, E);
  if (need > 0) ws = c.make({(int64_t)need}, at::kByte);
  check(lora_expert_rows(as<const int32_t>(ids), T, (int32_t)k, E, as<const int32_t>(slot),
                         as<int32_t>(row_token), as<int32_t>(positions), as<int32_t>(offsets),
                         as<int32_t>(row_slot), ptr(ws), need, c.stream()),
        "lora_expert_rows");
  return pack({&row_token, &positions, &offsets, row_slot ? &*row_slot : nullptr});
}

// (rows, positions, weights, residual or None, y or None) -> (y,)
PyObject* combine(PyObject* const* a) {
  Call c;
  const at::Tensor r = c.tensor(a[0], "rows"), pos = c.int32(a[1], "positions"),
                   w = c.tensor(a[2], "weights");
  const Opt res = c.optional(a[3], "residual"), y_in = c.optional(a[4], "y");
  if (r.dim() != 2 || pos.dim() != 2)
    refuse("rows must be [num_rows, width] and positions [T, top_k]");
  const int64_t T = pos.size(0), k = pos.size(1), width = r.size(1);
  if (k > INT32_MAX) refuse("positions must be [T, top_k]");
  given(w, T, k, at::kFloat, "weights");
  if (res) given(*res, T, width, r.scalar_type(), "residual");
  if (y_in) given(*y_in, T, width, r.scalar_type(), "y");
  const int dt = dtype_code(r.scalar_type());
  const c10::DeviceGuard guard(r.device());
  const at::Tensor y = y_in ? *y_in : c.make({T, width}, r.scalar_type());
  check(lora_combine_experts(dt, ptr(r), r.size(0), width, as<const int32_t>(pos),
                             as<const float>(w), T, (int32_t)k, ptr(res), ptr(y), c.stream()),
        "lora_combine_experts");
  return pack({&y});
}

// (form, x, row_index or None) -> (rows or None, codes, scales)
PyObject* quantize(PyObject* const* a) {
  Call c;
  const int32_t form = integer32(a[0], "form");
  const at::Tensor x = c.tensor(a[1], "x");
  Opt index;
  int64_t n = 0, K = 0, x_rows = 0;
  if (form == LORA_QUANTIZE_PLAIN) {
    if (x.dim() < 1) refuse("x must be [..., K]");
    K = x.size(-1);
    n = x_rows = K > 0 ? x.numel() / K : 0;
  } else if (form == LORA_QUANTIZE_GATHER) {
    index = c.int32(a[2], "row_token");
    if (x.dim() != 2 || index->dim() != 1) refuse("x must be [T, K] and row_token [rows]");
    n = index->numel();
    K = x.size(1);
    x_rows = x.size(0);
  } else {
    if (x.dim() != 2 || x.size(1) % 2) refuse("gate_up must be [rows, 2 K]");
    n = x_rows = x.size(0);
    K = x.size(1) / 2;
  }
  const int dt = dtype_code(x.scalar_type());
  const int64_t ld = lora_mxfp4_scale_row_bytes(K);
  if (ld == 0) refuse("K must be a multiple of 32, at most 2^20");
  const c10::DeviceGuard guard(x.device());
  const at::Tensor codes = c.make({n, K / 2}, at::kByte), scales = c.make({n, ld}, at::kByte);
  Opt out;
  if (form != LORA_QUANTIZE_PLAIN) out = c.make({n, K}, x.scalar_type());
  check(lora_quantize_mxfp4(dt, form, ptr(x), x_rows, as<const int32_t>(index), n, K, ptr(out),
                            as<uint8_t>(codes), as<uint8_t>(scales), c.stream()),
        "lora_quantize_mxfp4");
  return pack({out ? &*out : nullptr, &codes, &scales});
}

// (pair, dtype or None) -> (values [rows, K],)
PyObject* dequantize(PyObject* const* a) {
  Call c;
  const Held q = held(c, a[0], "dequantize_mxfp4");
  const at::ScalarType st = dtype_arg(a[1], at::kBFloat16);
  const int dt = dtype_code(st);
  const c10::DeviceGuard guard(q.codes.device());
  const at::Tensor out = c.make({q.rows, q.K}, st);
  check(lora_dequantize_mxfp4(dt, as<const uint8_t>(q.codes), as<const uint8_t>(q.scales), q.rows,
                              q.K, ptr(out), c.stream()),
        "lora_dequantize_mxfp4");
  return pack({&out});
}

// (x, w, offsets or None, dtype or None, y or None) -> (y,)
PyObject* linear(PyObject* const* a) {
  Call c;
  const bool grouped = a[2] != Py_None;
  const char* what = grouped ? "mxfp4_expert_linear" : "mxfp4_linear";
  const Held x = held(c, a[0], what), w = held(c, a[1], what);
  if (x.K != w.K || x.codes.dim() != 2 || w.codes.dim() != (grouped ? 3 : 2))
    refuse("%s: shape mismatch between x and w", what);
  Opt off;
  if (grouped) {
    off = c.int32(a[2], "offsets");
    if (off->numel() != w.codes.size(0) + 1 || off->numel() > INT32_MAX)
      refuse("%s: offsets must be [experts + 1]", what);
  }
  const int64_t N = w.codes.size(-2);
  const Opt y_in = c.optional(a[4], "y");
  const at::ScalarType st = dtype_arg(a[3], y_in ? y_in->scalar_type() : at::kBFloat16);
  if (y_in) given(*y_in, x.rows, N, st, "y");
  const int dt = dtype_code(st);
  const c10::DeviceGuard guard(x.codes.device());
  const at::Tensor y = y_in ? *y_in : c.make({x.rows, N}, st);
  if (grouped)
    check(lora_mxfp4_expert_linear(dt, as<const uint8_t>(x.codes), as<const uint8_t>(x.scales),
                                   x.rows, as<const uint8_t>(w.codes), as<const uint8_t>(w.scales),
                                   N, x.K, as<const int32_t>(off), (int32_t)w.codes.size(0),
                                   ptr(y), c.stream()),
          "lora_mxfp4_expert_linear");
  else
    check(lora_mxfp4_linear(dt, as<const uint8_t>(x.codes), as<const uint8_t>(x.scales), x.rows,
                            as<const uint8_t>(w.codes), as<const uint8_t>(w.scales), N, x.K,
                            ptr(y), c.stream()),
          "lora_mxfp4_linear");
  return pack({&y});
}

// A function of this file as Python calls it: its number of arguments, and
// what it throws (torch's and Python's errors keep their types).
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (LoraError, torch._C._cuda_getCurrentRawStream)
PyObject* setup(PyObject* const* a) {
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(g_stream, a[1]);
  Py_RETURN_NONE;
}

#define ENTRY(NAME, N) \
  { #NAME, (PyCFunction)(void*)entry<NAME, N>, METH_FASTCALL, nullptr }
PyMethodDef methods[] = {ENTRY(setup, 2),      ENTRY(route, 11),     ENTRY(rows, 3),
                         ENTRY(combine, 5),    ENTRY(quantize, 3),   ENTRY(dequantize, 2),
                         ENTRY(linear, 5),     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_experts", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__experts(void) { return PyModule_Create(&module); }
