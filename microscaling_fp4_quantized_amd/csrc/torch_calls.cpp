// The Python calls of the 8-bit and mixture-of-experts operators without their interpreter time: checks a call's tensors
// and enters the C ABI. A decode step makes many calls of a few microseconds, and checking eight tensors in
// Python and marshalling them through ctypes takes as long as such a call's kernel (norm of one row of 4096: 8.1 us a
// call through binding.py alone, 2.6 of them the kernel's).
//
// Every function takes the entry point's address, the current device, its stream and the operands, and returns the
// entry point's status, or None where the operands are not plainly right (another type, shape, stride or
// device than the contract's): binding.py then makes the same call its own way, and says what is wrong. Nothing is
// launched before None is returned.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <type_traits>

#include "../../include/fp4.h"

namespace {

using at::ScalarType;
using at::Tensor;

// A call's arguments, read in order; `good` turns false at the first that is not plainly right.
struct Args {
  PyObject* const* at;
  Py_ssize_t left;
  bool good = true;
  int64_t device = -1;

  PyObject* next() {
    if (left <= 0) {
      good = false;
      return Py_None;
    }
    --left;
    return *at++;
  }
  int64_t integer() {
    PyObject* o = next();
    if (!PyLong_CheckExact(o)) {
      good = false;
      return 0;
    }
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      good = false;
    }
    return v;
  }
  void* address() {
    PyObject* o = next();
    void* p = PyLong_CheckExact(o) ? PyLong_AsVoidPtr(o) : nullptr;
    if (PyErr_Occurred()) {
      PyErr_Clear();
      good = false;
    }
    return p;
  }
  double number() {
    PyObject* o = next();
    if (!PyFloat_CheckExact(o)) good = false;
    return good ? PyFloat_AS_DOUBLE(o) : 0.0;
  }
  bool truth() {
    PyObject* o = next();
    if (o != Py_True && o != Py_False) good = false;
    return o == Py_True;
  }
  // A tensor on the device; null where None is allowed and given, or where it is not plainly right.
  const Tensor* tensor(ScalarType type, int64_t dims, bool optional = false) {
    PyObject* o = next();
    if (optional && o == Py_None) return nullptr;
    if (!good || !THPVariable_Check(o)) {
      good = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.get_device() != device || t.scalar_type() != type || t.dim() != dims) {
      good = false;
      return nullptr;
    }
    return &t;
  }
  // A contiguous tensor of this shape.
  void* plain(ScalarType type, std::initializer_list<int64_t> shape, bool optional = false) {
    const Tensor* t = tensor(type, (int64_t)shape.size(), optional);
    if (t == nullptr) return nullptr;
    if (!t->is_contiguous() || !t->sizes().equals(at::IntArrayRef(shape))) {
      good = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  // Rows of bf16 with unit column stride.
  struct Rows {
    void* data;
    int64_t rows, cols, ld;
  };
  Rows bf16_rows(bool optional = false) {
    const Tensor* t = tensor(ScalarType::BFloat16, 2, optional);
    if (t == nullptr) return {nullptr, 0, 0, 0};
    if (t->stride(1) != 1) good = false;
    return {t->data_ptr(), t->size(0), t->size(1), t->size(0) > 1 ? t->stride(0) : t->size(1)};
  }
};

PyObject* answer(bool good, int status) {
  if (!good) Py_RETURN_NONE;
  return PyLong_FromLong(status);
}

constexpr int64_t kGroup = 128;

// quantize(entry, device, stream, x, rows per scale, codes, scales)
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  auto entry = reinterpret_cast<decltype(&fp8_quantize)>(a.address());
  static_assert(std::is_same<decltype(&fp8_quantize), decltype(&fp8_quantize_weights)>::value, "one call for both");
  a.device = a.integer();
  void* stream = a.address();
  const auto x = a.bf16_rows();
  const int64_t per = a.integer();
  if (!a.good || per < 1) Py_RETURN_NONE;
  void* codes = a.plain(ScalarType::Float8_e4m3fn, {x.rows, x.cols});
  void* scales = a.plain(ScalarType::Float, {(x.rows + per - 1) / per, x.cols / kGroup});
  const bool good = a.good && a.left == 0;
  return answer(good, good ? entry(x.data, x.rows, x.cols, x.ld, (uint8_t*)codes, (float*)scales, stream) : 0);
}

// norm(entry, device, stream, x, weight, residual, eps, codes, scales, sum, normed)
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  auto entry = reinterpret_cast<decltype(&fp8_add_rmsnorm_quantize)>(a.address());
  a.device = a.integer();
  void* stream = a.address();
  const auto x = a.bf16_rows();
  void* w = a.plain(ScalarType::BFloat16, {x.cols});
  const auto r = a.bf16_rows(true);
  if (r.data != nullptr && (r.rows != x.rows || r.cols != x.cols)) a.good = false;
  const double eps = a.number();
  void* codes = a.plain(ScalarType::Float8_e4m3fn, {x.rows, x.cols});
  void* scales = a.plain(ScalarType::Float, {x.rows, x.cols / kGroup});
  void* h = a.plain(ScalarType::BFloat16, {x.rows, x.cols}, true);
  void* y = a.plain(ScalarType::BFloat16, {x.rows, x.cols}, true);
  const bool good = a.good && a.left == 0;
  return answer(good, good ? entry(x.data, x.rows, x.cols, x.ld, r.data, r.ld, w, (float)eps, (uint8_t*)codes, (float*)scales,
                                   h, y, stream)
                           : 0);
}

// linear(entry, device, stream, xq, xs, wq, ws, y)
PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  auto entry = reinterpret_cast<decltype(&fp8_linear)>(a.address());
  a.device = a.integer();
  void* stream = a.address();
  const Tensor* xq = a.tensor(ScalarType::Float8_e4m3fn, 2);
  if (!a.good || !xq->is_contiguous()) Py_RETURN_NONE;
  const int64_t M = xq->size(0), K = xq->size(1);
  void* xs = a.plain(ScalarType::Float, {M, K / kGroup});
  const Tensor* wq = a.tensor(ScalarType::Float8_e4m3fn, 2);
  if (!a.good || !wq->is_contiguous() || wq->size(1) != K) Py_RETURN_NONE;
  const int64_t N = wq->size(0);
  void* ws = a.plain(ScalarType::Float, {(N + kGroup - 1) / kGroup, K / kGroup});
  void* y = a.plain(ScalarType::BFloat16, {M, N});
  const bool good = a.good && a.left == 0;
  return answer(good, good ? entry((const uint8_t*)xq->data_ptr(), (const float*)xs, (const uint8_t*)wq->data_ptr(),
                                   (const float*)ws, M, N, K, y, stream)
                           : 0);
}

// route(entry, device, stream, x, router, k, renormalize, ids, weights, workspace)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  auto entry = reinterpret_cast<decltype(&fp4_moe_route)>(a.address());
  a.device = a.integer();
  void* stream = a.address();
  const auto x = a.bf16_rows();
  const Tensor* w = a.tensor(ScalarType::BFloat16, 2);
  if (!a.good || !w->is_contiguous() || w->size(1) != x.cols) Py_RETURN_NONE;
  const int64_t k = a.integer();
  const bool renorm = a.truth();
  void* ids = a.plain(ScalarType::Int, {x.rows, k});
  void* p = a.plain(ScalarType::Float, {x.rows, k});
  const Tensor* ws = a.tensor(ScalarType::Byte, 1);
  if (!a.good || a.left != 0 || !ws->is_contiguous() || k > INT32_MAX || k < INT32_MIN) Py_RETURN_NONE;
  return answer(true, entry(x.data, x.rows, x.cols, x.ld, w->data_ptr(), w->size(0), (int)k, renorm, (int*)ids, (float*)p,
                            ws->data_ptr(), (size_t)ws->numel(), stream));
}

// experts(entry, device, stream, x, ids, weights, w13q, w13s, w2q, w2s, block, y, workspace)
PyObject* experts(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  auto entry = reinterpret_cast<decltype(&fp4_moe_experts)>(a.address());
  a.device = a.integer();
  void* stream = a.address();
  const auto x = a.bf16_rows();
  const Tensor* ids = a.tensor(ScalarType::Int, 2);
  if (!a.good || !ids->is_contiguous() || ids->size(0) != x.rows) Py_RETURN_NONE;
  const int64_t T = x.rows, D = x.cols, k = ids->size(1);
  void* p = a.plain(ScalarType::Float, {T, k});
  const Tensor* w13q = a.tensor(ScalarType::Byte, 3);
  if (!a.good || !w13q->is_contiguous() || w13q->size(1) % 2 != 0 || w13q->size(2) != D / 2) Py_RETURN_NONE;
  const int64_t E = w13q->size(0), I = w13q->size(1) / 2;
  void* w13s = a.plain(ScalarType::Byte, {E, 2 * I, D / 32});
  void* w2q = a.plain(ScalarType::Byte, {E, D, I / 2});
  void* w2s = a.plain(ScalarType::Byte, {E, D, I / 32});
  const int64_t block = a.integer();
  void* y = a.plain(ScalarType::BFloat16, {T, D});
  const Tensor* ws = a.tensor(ScalarType::Byte, 1);
  if (!a.good || a.left != 0 || !ws->is_contiguous() || D % 32 != 0 || I % 32 != 0 || k > INT32_MAX || block < 0 || block > 1024)
    Py_RETURN_NONE;
  return answer(true, entry(x.data, T, D, x.ld, (const int*)ids->data_ptr(), (const float*)p, (int)k, E, I, (int)block,
                            (const uint8_t*)w13q->data_ptr(), (const uint8_t*)w13s, (const uint8_t*)w2q, (const uint8_t*)w2s, y,
                            ws->data_ptr(), (size_t)ws->numel(), stream));
}

// A C++ exception of torch's must not leave through the interpreter's C frames.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (...) {
    Py_RETURN_NONE;
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method<quantize>("quantize"), method<norm>("norm"), method<linear>("linear"),
                          method<route>("route"), method<experts>("experts"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// ABI_VERSION: the header that the calls above were compiled against; binding.py enters no library of another.
PyMODINIT_FUNC PyInit__torch_calls(void) {
  PyObject* module = PyModule_Create(&kModule);
  if (module != nullptr && PyModule_AddIntConstant(module, "ABI_VERSION", FP4_ABI_VERSION) != 0) Py_CLEAR(module);
  return module;
}
