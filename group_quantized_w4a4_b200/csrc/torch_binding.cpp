// torch_binding.cpp -- the torch side of the block-scaled FP8, expert and block-norm calls: checks
// of tensors, outputs and workspaces from torch's caching allocator, and the call of the C entry
// point (include/apex_w4a4.h) on the current stream of the tensors' device.
//
// A decode step makes many calls whose kernels last a few microseconds.  Marshalling them in
// Python costs several times that (a block_norm call: 24.5 us in Python with ctypes, of which the
// launch is 3); here the whole call costs little more than its launches.
#include <Python.h>
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <optional>

#include "apex_w4a4.h"

namespace {

// The library's entry points, looked up once by bind().
struct Api {
  decltype(&apex_quantize_act_fp8_block) quantize;
  decltype(&apex_gemm_fp8_block) gemm;
  decltype(&apex_linear_fp8_block) linear;
  decltype(&apex_linear_fp8_block_workspace_size) linear_ws;
  decltype(&apex_route_experts) route;
  decltype(&apex_plan_experts) plan;
  decltype(&apex_route_plan_experts) route_plan;
  decltype(&apex_moe_mlp_fp8_block) moe;
  decltype(&apex_moe_mlp_fp8_block_workspace_size) moe_ws;
  decltype(&apex_block_norm) norm;
} api;
PyObject* apex_error = nullptr;

struct BadValue {};   // a Python ValueError has been set

[[noreturn]] void value_error(const char* name, const std::string& what) {
  PyErr_Format(PyExc_ValueError, "%s: %s", name, what.c_str());
  throw BadValue{};
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// Tensor arguments of one call, on one device.
struct Tensors {
  int device = -1;
  std::optional<c10::cuda::CUDAGuard> guard;

  const at::Tensor* take(PyObject* o, const char* name, bool optional = false) {
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) value_error(name, "expected a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) value_error(name, "expected a CUDA tensor (device memory)");
    if (!t.is_contiguous()) value_error(name, "expected a contiguous tensor");
    const int d = t.get_device();
    if (device < 0) {
      device = d;
      if (d != c10::cuda::current_device()) guard.emplace(d);
    } else if (d != device) {
      value_error(name, "expected tensors on one device");
    }
    return &t;
  }
  // of a given type (nullopt: not checked) and shape
  const at::Tensor* take(PyObject* o, const char* name, std::optional<at::ScalarType> type,
                         std::initializer_list<int64_t> shape, bool optional = false) {
    const at::Tensor* t = take(o, name, optional);
    if (t) expect(*t, name, type, shape);
    return t;
  }
  static void expect(const at::Tensor& t, const char* name, std::optional<at::ScalarType> type,
                     std::initializer_list<int64_t> shape) {
    if (type && t.scalar_type() != *type)
      value_error(name, std::string("expected ") + c10::toString(*type) + ", got " +
                            c10::toString(t.scalar_type()));
    if (t.sizes() != at::IntArrayRef(shape))
      value_error(name, "expected shape " + shape_text(at::IntArrayRef(shape)) + ", got " +
                            shape_text(t.sizes()));
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    // (not through the dispatcher, which costs 0.5 us a tensor)
    return at::Tensor(at::detail::empty_cuda(shape, type, c10::Device(at::kCUDA, (c10::DeviceIndex)device),
                                             std::nullopt));
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

const at::Tensor& matrix(const at::Tensor* t, const char* name, int64_t dims) {
  if (t->dim() != dims) value_error(name, "expected " + std::to_string(dims) + " dimensions");
  return *t;
}

int32_t dtype_code(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kHalf: return APEX_DTYPE_F16;
    case at::kBFloat16: return APEX_DTYPE_BF16;
    case at::kFloat: return APEX_DTYPE_F32;
    default: value_error(name, std::string("expected fp16, bf16 or fp32, got ") +
                                   c10::toString(t.scalar_type()));
  }
}

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
int64_t groups_of(int64_t n) { return (n + 127) / 128; }

struct Failed {};   // an ApexError has been set
void check(apex_status_t st, const char* where) {
  if (st == APEX_OK) return;
  PyObject* args = Py_BuildValue("(is)", (int)st, where);
  if (args) {
    PyErr_SetObject(apex_error, args);
    Py_DECREF(args);
  }
  throw Failed{};
}

int64_t as_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  (void)name;
  return v;
}
int32_t as_int32(PyObject* o, const char* name) {
  const int64_t v = as_int(o, name);
  if (v != (int32_t)v) value_error(name, "out of range");
  return (int32_t)v;
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed{};
  return (float)v;
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Failed{};
  return v != 0;
}

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

template <typename... Ts>
PyObject* tuple_of(const Ts&... ts) {
  PyObject* items[] = {wrap(ts)...};
  PyObject* r = PyTuple_New(sizeof...(ts));
  for (size_t i = 0; i < sizeof...(ts); ++i) {
    if (!r || !items[i]) {
      for (PyObject* p : items) Py_XDECREF(p);
      if (r) Py_DECREF(r);
      return nullptr;
    }
  }
  for (size_t i = 0; i < sizeof...(ts); ++i) PyTuple_SET_ITEM(r, (Py_ssize_t)i, items[i]);
  return r;
}

// Runs f with C++ exceptions turned into Python ones; the arguments' number is fixed by the
// Python wrappers.
template <int N, typename F>
PyObject* guarded(Py_ssize_t n, F&& f) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %d", N, (int)n);
    return nullptr;
  }
  if (!apex_error) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
    return nullptr;
  }
  try {
    return f();
  } catch (const BadValue&) {
    return nullptr;
  } catch (const Failed&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ the calls

// (x) -> codes, scales
PyObject* quantize_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<1>(n, [&]() -> PyObject* {
    Tensors ts;
    const at::Tensor& x = matrix(ts.take(a[0], "x"), "x", 2);
    const int64_t M = x.size(0), K = x.size(1);
    const int32_t dt = dtype_code(x, "x");
    at::Tensor codes = ts.empty({M, K}, at::kByte), scales = ts.empty({M, groups_of(K)}, at::kFloat);
    if (M)
      check(api.quantize(x.data_ptr(), dt, M, K, codes.data_ptr(), scales.data_ptr(), ts.stream()),
            "apex_quantize_act_fp8_block");
    return tuple_of(codes, scales);
  });
}

// (a_codes, a_scales, w_codes, w_scales, bf16, out) -> y
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<6>(n, [&]() -> PyObject* {
    Tensors ts;
    const at::Tensor& ac = matrix(ts.take(a[0], "a_codes"), "a_codes", 2);
    const at::Tensor& wc = matrix(ts.take(a[2], "w_codes"), "w_codes", 2);
    const int64_t M = ac.size(0), K = ac.size(1), N = wc.size(0), G = groups_of(K);
    Tensors::expect(ac, "a_codes", at::kByte, {M, K});
    Tensors::expect(wc, "w_codes", at::kByte, {N, K});
    const at::Tensor* as = ts.take(a[1], "a_scales", at::kFloat, {M, G});
    const at::Tensor* ws = ts.take(a[3], "w_scales", at::kFloat, {groups_of(N), G});
    const at::Tensor* out = ts.take(a[5], "out", std::nullopt, {M, N}, true);
    at::Tensor y = out ? *out : ts.empty({M, N}, as_bool(a[4]) ? at::kBFloat16 : at::kHalf);
    const int32_t dt = dtype_code(y, "out");
    if (M)
      check(api.gemm(M, N, K, ac.data_ptr(), as->data_ptr(), wc.data_ptr(), ws->data_ptr(), dt,
                     y.data_ptr(), ts.stream()),
            "apex_gemm_fp8_block");
    return wrap(y);
  });
}

// (x, w_codes, w_scales, out) -> y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<4>(n, [&]() -> PyObject* {
    Tensors ts;
    const at::Tensor& x = matrix(ts.take(a[0], "x"), "x", 2);
    const at::Tensor& wc = matrix(ts.take(a[1], "w_codes"), "w_codes", 2);
    const int64_t M = x.size(0), K = x.size(1), N = wc.size(0);
    Tensors::expect(wc, "w_codes", at::kByte, {N, K});
    const at::Tensor* ws = ts.take(a[2], "w_scales", at::kFloat, {groups_of(N), groups_of(K)});
    const at::Tensor* out = ts.take(a[3], "out", x.scalar_type(), {M, N}, true);
    const int32_t dt = dtype_code(x, "x");
    at::Tensor y = out ? *out : ts.empty({M, N}, x.scalar_type());
    if (M) {
      const size_t bytes = api.linear_ws(M, N, K);
      at::Tensor w = ts.empty({(int64_t)(bytes ? bytes : 1)}, at::kByte);
      check(api.linear(M, N, K, x.data_ptr(), dt, wc.data_ptr(), ws->data_ptr(), y.data_ptr(),
                       w.data_ptr(), bytes, ts.stream()),
            "apex_linear_fp8_block");
    }
    return wrap(y);
  });
}

// (logits, k, bias, score, groups, topk_groups, renormalize, scale, mask, plan)
//   -> weights, ids (, offsets, order)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<10>(n, [&]() -> PyObject* {
    Tensors ts;
    const at::Tensor& z = matrix(ts.take(a[0], "logits"), "logits", 2);
    const int64_t T = z.size(0), E = z.size(1);
    const int32_t k = as_int32(a[1], "k");
    const at::Tensor* bias = ts.take(a[2], "bias", at::kFloat, {E}, true);
    const at::Tensor* mask = ts.take(a[8], "mask", at::kBool, {T}, true);
    const int32_t dt = dtype_code(z, "logits");
    const bool plan = as_bool(a[9]);
    if (k < 0 || E > INT32_MAX) value_error("k", "out of range");
    at::Tensor w = ts.empty({T, k}, at::kFloat), ids = ts.empty({T, k}, at::kInt), offsets, order;
    if (plan) {
      offsets = ts.empty({E + 1}, at::kInt);
      order = ts.empty({T * k}, at::kInt);
    }
    if (T) {
      const int32_t score = as_int32(a[3], "score"), G = as_int32(a[4], "groups");
      const int32_t TG = as_int32(a[5], "topk_groups"), renorm = as_bool(a[6]);
      const float scale = as_float(a[7]);
      if (plan)
        check(api.route_plan(z.data_ptr(), dt, T, (int32_t)E, k, score, ptr(bias), G, TG, renorm,
                             scale, ptr(mask), w.data_ptr(), ids.data_ptr(), offsets.data_ptr(),
                             order.data_ptr(), ts.stream()),
              "apex_route_plan_experts");
      else
        check(api.route(z.data_ptr(), dt, T, (int32_t)E, k, score, ptr(bias), G, TG, renorm, scale,
                        ptr(mask), w.data_ptr(), ids.data_ptr(), ts.stream()),
              "apex_route_experts");
    } else if (plan) {
      offsets.zero_();
    }
    return plan ? tuple_of(w, ids, offsets, order) : tuple_of(w, ids);
  });
}

// (ids, experts) -> offsets, order
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<2>(n, [&]() -> PyObject* {
    Tensors ts;
    const at::Tensor& ids = matrix(ts.take(a[0], "ids"), "ids", 2);
    const int64_t T = ids.size(0), k = ids.size(1);
    Tensors::expect(ids, "ids", at::kInt, {T, k});
    const int32_t E = as_int32(a[1], "experts");
    if (E < 1 || k > INT32_MAX) value_error("experts", "out of range");
    at::Tensor offsets = ts.empty({(int64_t)E + 1}, at::kInt), order = ts.empty({T * k}, at::kInt);
    if (T)
      check(api.plan(ids.data_ptr(), T, (int32_t)k, E, offsets.data_ptr(), order.data_ptr(),
                     ts.stream()),
            "apex_plan_experts");
    else
      offsets.zero_();
    return tuple_of(offsets, order);
  });
}

// (x, weights, ids, offsets, order, w13_codes, w13_scales, w2_codes, w2_scales, out) -> y
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<10>(n, [&]() -> PyObject* {
    Tensors ts;
    const at::Tensor& x = matrix(ts.take(a[0], "x"), "x", 2);
    const at::Tensor& ids = matrix(ts.take(a[2], "ids"), "ids", 2);
    const at::Tensor& w13 = matrix(ts.take(a[5], "w13_codes"), "w13_codes", 4);
    const int64_t T = x.size(0), H = x.size(1), k = ids.size(1), E = w13.size(0), I = w13.size(2);
    const int64_t GH = groups_of(H), GI = groups_of(I);
    const at::Tensor* wt = ts.take(a[1], "weights", at::kFloat, {T, k});
    Tensors::expect(ids, "ids", at::kInt, {T, k});
    const at::Tensor* off = ts.take(a[3], "offsets", at::kInt, {E + 1});
    const at::Tensor* order = ts.take(a[4], "order", at::kInt, {T * k});
    Tensors::expect(w13, "w13_codes", at::kByte, {E, 2, I, H});
    const at::Tensor* s13 = ts.take(a[6], "w13_scales", at::kFloat, {E, 2, GI, GH});
    const at::Tensor* w2 = ts.take(a[7], "w2_codes", at::kByte, {E, H, I});
    const at::Tensor* s2 = ts.take(a[8], "w2_scales", at::kFloat, {E, GH, GI});
    const at::Tensor* out = ts.take(a[9], "out", x.scalar_type(), {T, H}, true);
    const int32_t dt = dtype_code(x, "x");
    if (E > INT32_MAX || k > INT32_MAX) value_error("w13_codes", "out of range");
    at::Tensor y = out ? *out : ts.empty({T, H}, x.scalar_type());
    if (T) {
      const size_t bytes = api.moe_ws(T, (int32_t)E, (int32_t)k, H, I);
      at::Tensor w = ts.empty({(int64_t)(bytes ? bytes : 1)}, at::kByte);
      check(api.moe(T, (int32_t)E, (int32_t)k, H, I, x.data_ptr(), dt, wt->data_ptr(),
                    ids.data_ptr(), off->data_ptr(), order->data_ptr(), w13.data_ptr(),
                    s13->data_ptr(), w2->data_ptr(), s2->data_ptr(), y.data_ptr(), w.data_ptr(),
                    bytes, ts.stream()),
            "apex_moe_mlp_fp8_block");
    }
    return wrap(y);
  });
}

// (x, pre_weight, residual, post_weight, gate, alpha, eps, weight_offset, values, codes)
//   -> h, y, codes, scales
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<10>(n, [&]() -> PyObject* {
    Tensors ts;
    const at::Tensor& x = matrix(ts.take(a[0], "x"), "x", 2);
    const int64_t T = x.size(0), H = x.size(1);
    const at::ScalarType t = x.scalar_type();
    const at::Tensor* pre = ts.take(a[1], "pre_weight", t, {H}, true);
    const at::Tensor* residual = ts.take(a[2], "residual", t, {T, H}, true);
    const at::Tensor* post = ts.take(a[3], "post_weight", t, {H}, true);
    const at::Tensor* gate = ts.take(a[4], "gate", true);
    int64_t rows = 0;
    if (gate) {
      rows = matrix(gate, "gate", 2).size(0);
      Tensors::expect(*gate, "gate", t, {rows, H});
    }
    const int32_t dt = dtype_code(x, "x");
    const bool want_y = as_bool(a[8]), want_codes = as_bool(a[9]);
    at::Tensor h = ts.empty({T, H}, t), y, codes, scales;
    if (want_y) y = ts.empty({T, H}, t);
    if (want_codes) {
      codes = ts.empty({T, H}, at::kByte);
      scales = ts.empty({T, groups_of(H)}, at::kFloat);
    }
    if (T)
      check(api.norm(x.data_ptr(), dt, T, H, ptr(residual), ptr(post), ptr(gate), rows,
                     as_float(a[5]), ptr(pre), as_float(a[6]), as_float(a[7]), h.data_ptr(),
                     want_y ? y.data_ptr() : nullptr, want_codes ? codes.data_ptr() : nullptr,
                     want_codes ? scales.data_ptr() : nullptr, ts.stream()),
            "apex_block_norm");
    return tuple_of(h, y, codes, scales);
  });
}

// (addresses of the entry points in Api's order, the ApexError class)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = sizeof(Api) / sizeof(void*);
  if (n != kEntries + 1) {
    PyErr_SetString(PyExc_TypeError, "bind: wrong number of entry points");
    return nullptr;
  }
  void* p[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null entry point");
      return nullptr;
    }
  }
  memcpy(&api, p, sizeof(api));
  Py_INCREF(a[kEntries]);
  apex_error = a[kEntries];
  Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind),  ENTRY(quantize_act), ENTRY(gemm), ENTRY(linear),
                         ENTRY(route), ENTRY(plan),         ENTRY(moe),  ENTRY(norm),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "apex_torch", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_apex_torch() { return PyModule_Create(&module_def); }
