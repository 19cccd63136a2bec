// The Python calls of the 8-bit, mixture-of-experts and attention operators without their interpreter time: checks a call's tensors
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
  // A tensor on the device of any type; null where None is allowed and given, or where it is not plainly right.
  const Tensor* any(int64_t dims, bool optional = false) {
    PyObject* o = next();
    if (optional && o == Py_None) return nullptr;
    if (!good || !THPVariable_Check(o)) {
      good = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.get_device() != device || t.dim() != dims) {
      good = false;
      return nullptr;
    }
    return &t;
  }
  // Rows of heads of bf16 whose numbers lie together; a stride of a dimension of one is any that suits.
  struct Heads {
    void* data;
    int64_t rows, heads, dim, row, head;
  };
  Heads bf16_heads(bool optional = false) {
    const Tensor* t = any(3, optional);
    if (t == nullptr) return {nullptr, 0, 0, 0, 0, 0};
    if (t->scalar_type() != ScalarType::BFloat16 || t->stride(2) != 1) good = false;
    const int64_t T = t->size(0), H = t->size(1), D = t->size(2);
    return {t->data_ptr(), T, H, D, T > 1 ? t->stride(0) : H * D, H > 1 ? t->stride(1) : D};
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

// Strides of pages, heads and tokens.
void strides_of(const Tensor& t, int64_t least, int64_t* to) {
  for (int i = 0; i < 3; ++i) to[i] = t.size(i) > 1 ? t.stride(i) : (least > 1 ? least : 1);
}

// k_pages, v_pages, table, lengths, k_scales, v_scales -> the cache's description.
fp4_kv_cache cache_of(Args& a) {
  fp4_kv_cache c{};
  const Tensor *k = a.any(4), *v = a.any(4);
  const Tensor* table = a.tensor(ScalarType::Int, 2);
  if (!a.good) return c;
  const bool e4m3 = k->scalar_type() == ScalarType::Float8_e4m3fn;
  int64_t ks[3], vs[3];
  strides_of(*k, k->size(3), ks);
  strides_of(*v, v->size(3), vs);
  const int64_t page = k->size(2), dim = k->size(3), heads = k->size(1), B = table->size(0), cols = table->size(1);
  a.good = (e4m3 || k->scalar_type() == ScalarType::BFloat16) && v->scalar_type() == k->scalar_type() && v->sizes() == k->sizes() &&
           ks[0] == vs[0] && ks[1] == vs[1] && ks[2] == vs[2] && k->stride(3) == 1 && v->stride(3) == 1 &&
           (cols <= 1 || table->stride(1) == 1) && heads <= 1024 && dim <= 1024 && page <= 1024;
  c.lengths = (const int*)a.plain(ScalarType::Int, {B});
  const Tensor *sk = a.any(3, !e4m3), *sv = a.any(3, !e4m3);
  if (!a.good) return c;
  if (e4m3) {
    int64_t x[3], y[3];
    strides_of(*sk, 1, x);
    strides_of(*sv, 1, y);
    const auto shape = k->sizes().slice(0, 3);
    a.good = sk->scalar_type() == ScalarType::Float && sv->scalar_type() == ScalarType::Float && sk->sizes() == shape &&
             sv->sizes() == shape && x[0] == y[0] && x[1] == y[1] && x[2] == y[2];
    c.k_scales = (float*)sk->data_ptr();
    c.v_scales = (float*)sv->data_ptr();
    c.scale_page_stride = x[0];
    c.scale_head_stride = x[1];
    c.scale_token_stride = x[2];
  } else if (sk != nullptr || sv != nullptr) {
    a.good = false;
  }
  c.k = k->data_ptr();
  c.v = v->data_ptr();
  c.pages = k->size(0);
  c.page_stride = ks[0];
  c.head_stride = ks[1];
  c.token_stride = ks[2];
  c.table = (const int*)table->data_ptr();
  c.table_stride = B > 1 ? table->stride(0) : cols;
  c.cols = cols;
  c.batch = B;
  c.dtype = e4m3 ? FP4_KV_E4M3 : FP4_KV_BF16;
  c.heads = (int)heads;
  c.dim = (int)dim;
  c.page_size = (int)page;
  return c;
}

// append(entry, device, stream, k, v, k_pages, v_pages, table, lengths, k_scales, v_scales, starts, q, freqs, positions, axes,
// interleaved, out)
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  auto entry = reinterpret_cast<decltype(&fp4_kv_append)>(a.address());
  a.device = a.integer();
  void* stream = a.address();
  const auto k = a.bf16_heads(), v = a.bf16_heads();
  if (!a.good) Py_RETURN_NONE;
  const fp4_kv_cache c = cache_of(a);
  if (!a.good || k.heads != c.heads || k.dim != c.dim || v.rows != k.rows || v.heads != k.heads || v.dim != k.dim) Py_RETURN_NONE;
  const int64_t T = k.rows;
  const void* starts = a.plain(ScalarType::Int, {c.batch + 1}, true);
  if (a.good && starts == nullptr && T != c.batch) Py_RETURN_NONE;
  const auto q = a.bf16_heads(true);
  const Tensor* freqs = a.any(1, true);
  if (!a.good) Py_RETURN_NONE;
  const int64_t half = freqs != nullptr ? freqs->size(0) : 0;
  if (freqs != nullptr && (freqs->scalar_type() != ScalarType::Float || !freqs->is_contiguous() || half > 512)) Py_RETURN_NONE;
  // the two shapes of positions
  PyObject* p = a.left > 0 ? *a.at : nullptr;
  const bool flat = p != nullptr && THPVariable_Check(p) && THPVariable_Unpack(p).dim() == 1;
  const Tensor* positions = a.any(flat ? 1 : 2, true);
  if (!a.good) Py_RETURN_NONE;
  const int64_t n_axes = positions == nullptr ? 0 : flat ? 1 : positions->size(0);
  if (positions != nullptr && (positions->scalar_type() != ScalarType::Int || !positions->is_contiguous() || positions->numel() != n_axes * T ||
                               n_axes < 1 || n_axes > 1024))
    Py_RETURN_NONE;
  const void* axes = a.plain(ScalarType::Int, {half}, true);
  const bool interleaved = a.truth();
  const auto out = a.bf16_heads(true);
  if (!a.good || a.left != 0 || q.heads > 1024 || (q.data == nullptr) != (out.data == nullptr)) Py_RETURN_NONE;
  if (q.data != nullptr && (q.rows != T || q.dim != k.dim || out.rows != T || out.heads != q.heads || out.dim != q.dim)) Py_RETURN_NONE;
  if (freqs == nullptr && (q.data != nullptr || positions != nullptr || axes != nullptr)) Py_RETURN_NONE;
  if (positions == nullptr && axes != nullptr) Py_RETURN_NONE;
  const bool same = q.data == out.data;  // in place: strides that say nothing are the same ones
  return answer(true, entry(&c, (const int*)starts, T, k.data, k.row, k.head, v.data, v.row, v.head, q.data, q.row, q.head, (int)q.heads,
                            out.data, same && T == 1 ? q.row : out.row, same && q.heads == 1 ? q.head : out.head,
                            freqs != nullptr ? (const float*)freqs->data_ptr() : nullptr, (int)(2 * half), interleaved,
                            positions != nullptr ? (const int*)positions->data_ptr() : nullptr, (const int*)axes, (int)n_axes, stream));
}

// What the two attention calls share: q, k_pages, v_pages, table, lengths, k_scales, v_scales.
struct Query {
  Args::Heads q;
  fp4_kv_cache cache;
};
Query query_of(Args& a) {
  Query x{};
  x.q = a.bf16_heads();
  if (!a.good) return x;
  x.cache = cache_of(a);
  if (a.good && (x.q.dim != x.cache.dim || x.q.heads > 1024 || x.q.heads < 1 || x.cache.heads < 1 || x.q.heads % x.cache.heads != 0))
    a.good = false;
  return x;
}
// The rest of them: scale, window, sinks, out, workspace.
struct Rest {
  float scale;
  int64_t window, sinks, bytes;
  void *out, *workspace;
};
Rest rest_of(Args& a, const Query& x) {
  Rest r{};
  r.scale = (float)a.number();
  r.window = a.integer();
  r.sinks = a.integer();
  r.out = a.plain(ScalarType::BFloat16, {x.q.rows, x.q.heads, x.q.dim});
  const Tensor* ws = a.tensor(ScalarType::Byte, 1);
  if (!a.good || a.left != 0 || !ws->is_contiguous()) {
    a.good = false;
    return r;
  }
  r.workspace = ws->data_ptr();
  r.bytes = ws->numel();
  return r;
}

// decode(entry, device, stream, q, the cache's six, scale, window, sinks, out, workspace)
PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  auto entry = reinterpret_cast<decltype(&fp4_attention_decode)>(a.address());
  a.device = a.integer();
  void* stream = a.address();
  const Query x = query_of(a);
  if (!a.good || x.q.rows != x.cache.batch) Py_RETURN_NONE;
  const Rest r = rest_of(a, x);
  if (!a.good) Py_RETURN_NONE;
  return answer(true, entry(&x.cache, x.q.data, x.q.row, x.q.head, (int)x.q.heads, r.scale, r.window, r.sinks, r.out, r.workspace,
                            (size_t)r.bytes, stream));
}

// prompt(entry, device, stream, q, the cache's six, starts, scale, window, sinks, out, workspace)
PyObject* prompt(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  auto entry = reinterpret_cast<decltype(&fp4_attention_prompt)>(a.address());
  a.device = a.integer();
  void* stream = a.address();
  const Query x = query_of(a);
  if (!a.good) Py_RETURN_NONE;
  const void* starts = a.plain(ScalarType::Int, {x.cache.batch + 1});
  const Rest r = rest_of(a, x);
  if (!a.good) Py_RETURN_NONE;
  return answer(true, entry(&x.cache, (const int*)starts, x.q.rows, x.q.data, x.q.row, x.q.head, (int)x.q.heads, r.scale, r.window,
                            r.sinks, r.out, r.workspace, (size_t)r.bytes, stream));
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
                          method<route>("route"), method<experts>("experts"),
                          method<append>("append"), method<decode>("decode"), method<prompt>("prompt"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// ABI_VERSION: the header that the calls above were compiled against; binding.py enters no library of another.
PyMODINIT_FUNC PyInit__torch_calls(void) {
  PyObject* module = PyModule_Create(&kModule);
  if (module != nullptr && PyModule_AddIntConstant(module, "ABI_VERSION", FP4_ABI_VERSION) != 0) Py_CLEAR(module);
  return module;
}
