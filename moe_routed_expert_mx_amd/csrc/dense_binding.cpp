// dense_binding.cpp -- the short way from Python to the entry points of the dense side and of the block-scaled FP8 layer.
//
// A decode step's kernels take 3 to 6 us, and so do the checks and argument conversions of a
// ctypes call.  Each function here takes what its namesake in _lib.py takes (options as plain
// numbers), checks it the same way and calls the library on the current stream of the tensors'
// GPU.  It returns the library's status, or kNotTaken if it did not call it -- a tensor it does not
// like, another GPU than the current one --: those are left to _lib.py, which checks again and says
// what is wrong.  No function of the library is linked: their addresses come through bind().
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "moe_mx.h"

namespace {

decltype(&moe_gate) g_gate;
decltype(&moe_route) g_route;
decltype(&moe_quant_i8) g_quant;
decltype(&moe_linear_i8) g_linear;
decltype(&moe_rms_norm) g_norm;
decltype(&moe_quant_f8) g_quant_f8;
decltype(&moe_linear_f8) g_linear_f8;
decltype(&moe_lists) g_lists;
decltype(&moe_grouped_f8) g_grouped_f8;
PyObject* g_raw_stream;  // torch._C._cuda_getCurrentRawStream
PyObject* g_device;      // torch._C._cuda_getDevice

constexpr long kNotTaken = -100;

// The tensors of one call: each accessor clears `ok` if its tensor does not fit.
struct Call {
  bool ok = true;
  int device = -1;

  const at::Tensor* tensor(PyObject* o) {
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    const c10::Device d = t.device();
    if (device < 0) device = d.index();
    if (!d.is_cuda() || d.index() != device || device < 0) ok = false;
    return &t;
  }
  // A matrix whose rows are contiguous; -1 sizes are taken as they are and returned.
  void* matrix(PyObject* o, int64_t& rows, int64_t& cols, int64_t& ld) {
    const at::Tensor* t = tensor(o);
    if (!ok || t->dim() != 2) return fail();
    if (rows < 0) rows = t->size(0);
    if (cols < 0) cols = t->size(1);
    if (t->size(0) != rows || t->size(1) != cols || (t->stride(1) != 1 && cols != 1)) return fail();
    ld = rows == 1 ? cols : t->stride(0);
    if (ld < cols || rows > INT32_MAX || cols > INT32_MAX) return fail();
    return t->data_ptr();
  }
  float* vector(PyObject* o, int64_t n) {
    const at::Tensor* t = tensor(o);
    if (!ok || t->dim() != 1 || t->size(0) != n || (n != 1 && t->stride(0) != 1) || t->scalar_type() != at::kFloat)
      return static_cast<float*>(fail());
    return static_cast<float*>(t->data_ptr());
  }
  // Contiguous int32 [n]; -1: any, returned.
  int32_t* list(PyObject* o, int64_t& n) {
    const at::Tensor* t = tensor(o);
    if (!ok || t->dim() != 1 || (n >= 0 && t->size(0) != n) || (t->size(0) > 1 && t->stride(0) != 1) ||
        t->scalar_type() != at::kInt)
      return static_cast<int32_t*>(fail());
    n = t->size(0);
    return static_cast<int32_t*>(t->data_ptr());
  }
  // FP32 scales of blocks of rows: [.., rows, cols] contiguous, n numbers in all.
  float* blocks(PyObject* o, int64_t experts, int64_t rows, int64_t cols) {
    const at::Tensor* t = tensor(o);
    const int64_t d = experts < 0 ? 2 : 3;
    if (!ok || t->dim() != d || (d == 3 && t->size(0) != experts) || t->size(d - 2) != rows || t->size(d - 1) != cols ||
        !t->is_contiguous() || t->scalar_type() != at::kFloat)
      return static_cast<float*>(fail());
    return static_cast<float*>(t->data_ptr());
  }
  void* fail() {
    ok = false;
    return nullptr;
  }
  void need(bool b) { ok = ok && b; }
  // The stream of the tensors' GPU, which must be the current one.  The last step before the library's call: an
  // argument or an answer that was no number clears `ok` here.
  void* stream() {
    if (!ok || PyErr_Occurred()) return fail();
    PyObject* d = PyObject_CallNoArgs(g_device);
    const long current = d ? PyLong_AsLong(d) : -1;
    Py_XDECREF(d);
    if (current != device) return fail();
    PyObject* arg = PyLong_FromLong(device);
    PyObject* s = arg ? PyObject_CallOneArg(g_raw_stream, arg) : nullptr;
    Py_XDECREF(arg);
    if (!s) return fail();
    void* raw = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return PyErr_Occurred() ? fail() : raw;
  }
};

int type_of(PyObject* o) {
  switch (THPVariable_Unpack(o).scalar_type()) {
    case at::kBFloat16: return MOE_BF16;
    case at::kHalf: return MOE_F16;
    case at::kFloat: return MOE_F32;
    default: return -1;
  }
}
bool is(PyObject* o, at::ScalarType t) { return THPVariable_Unpack(o).scalar_type() == t; }

// gate(handle address, D, E, x, logits[, the tensor that holds the packed weight, or None])
long gate(PyObject* const* v, Py_ssize_t n) {
  Call c;
  const void* h = PyLong_AsVoidPtr(v[0]);
  int64_t B = -1, D = PyLong_AsLongLong(v[1]), E = PyLong_AsLongLong(v[2]), ldx = 0, ldl = 0;
  void* x = c.matrix(v[3], B, D, ldx);
  void* out = c.matrix(v[4], B, E, ldl);
  c.need(c.ok && is(v[3], at::kBFloat16) && is(v[4], at::kFloat));
  if (n > 5 && v[5] != Py_None) c.tensor(v[5]);
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  return g_gate(static_cast<const moe_gate_t*>(h), x, ldx, static_cast<int32_t>(B), static_cast<float*>(out), ldl, st);
}

// route(logits, ids, weights, score, bias, groups, topk_groups, group_score, renorm, scale)
long route(PyObject* const* v, Py_ssize_t) {
  Call c;
  int64_t B = -1, E = -1, K = -1, ldl = 0, ld = 0;
  void* logits = c.matrix(v[0], B, E, ldl);
  void* ids = c.matrix(v[1], B, K, ld);
  c.need(ld == K);
  void* weights = c.matrix(v[2], B, K, ld);
  c.need(ld == K);
  c.need(c.ok && type_of(v[0]) >= 0 && is(v[1], at::kInt) && is(v[2], at::kFloat));
  const float* bias = v[4] == Py_None ? nullptr : c.vector(v[4], E);
  const long score = PyLong_AsLong(v[3]), groups = PyLong_AsLong(v[5]), kept = PyLong_AsLong(v[6]),
             ranked = PyLong_AsLong(v[7]);
  const int renorm = PyObject_IsTrue(v[8]);
  const float scale = static_cast<float>(PyFloat_AsDouble(v[9]));
  // (the library reads a scale of 0 as 1)
  c.need(renorm >= 0 && scale != 0.0f && std::isfinite(scale) && groups >= 0 && groups <= 64 && kept >= 0 && kept <= 64);
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  const moe_route_opts_t o = {static_cast<int32_t>(score),  static_cast<int32_t>(groups), static_cast<int32_t>(kept),
                              static_cast<int32_t>(ranked), renorm, scale, bias, {0, 0}};
  return g_route(logits, type_of(v[0]), ldl, static_cast<int32_t>(B), static_cast<int32_t>(E), static_cast<int32_t>(K), &o,
                 static_cast<int32_t*>(ids), static_cast<float*>(weights), st);
}

// quant(x, codes, scales)
long quant(PyObject* const* v, Py_ssize_t) {
  Call c;
  int64_t M = -1, K = -1, ldx = 0, ldc = 0;
  void* x = c.matrix(v[0], M, K, ldx);
  void* codes = c.matrix(v[1], M, K, ldc);
  float* scales = c.vector(v[2], M);
  c.need(c.ok && type_of(v[0]) >= 0 && is(v[1], at::kChar));
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  return g_quant(x, type_of(v[0]), ldx, static_cast<int32_t>(M), static_cast<int32_t>(K), static_cast<int8_t*>(codes), ldc,
                 scales, st);
}

// linear(a, a_scales, w, w_scales, out, act, bias, add)
long linear(PyObject* const* v, Py_ssize_t) {
  Call c;
  int64_t M = -1, K = -1, N = -1, lda = 0, ldw = 0, ldo = 0;
  const long act = PyLong_AsLong(v[5]);
  void* a = c.matrix(v[0], M, K, lda);
  void* w = c.matrix(v[2], N, K, ldw);
  int64_t cols = act == 1 ? N / 2 : N;
  c.need((act == 0 || act == 1) && !(act == 1 && N % 2));
  void* out = c.matrix(v[4], M, cols, ldo);
  const float* sa = c.vector(v[1], M);
  const float* sw = c.vector(v[3], N);
  c.need(c.ok && is(v[0], at::kChar) && is(v[2], at::kChar) && type_of(v[4]) >= 0);
  moe_linear_opts_t o = {static_cast<int32_t>(act), 0, nullptr, nullptr, 0};
  if (v[6] != Py_None) o.bias_dev = c.vector(v[6], N);
  if (v[7] != Py_None) {
    o.add_dev = c.matrix(v[7], M, cols, o.ldadd);
    c.need(c.ok && type_of(v[7]) == type_of(v[4]));
  }
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  return g_linear(static_cast<const int8_t*>(a), lda, sa, static_cast<const int8_t*>(w), ldw, sw, static_cast<int32_t>(M),
                  static_cast<int32_t>(N), static_cast<int32_t>(K), &o, out, type_of(v[4]), ldo, st);
}

constexpr at::ScalarType kE4m3 = at::kFloat8_e4m3fn;
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// quant_f8(x, codes, scales)
long quant_f8(PyObject* const* v, Py_ssize_t) {
  Call c;
  int64_t M = -1, K = -1, ldx = 0, ldc = 0, lds = 0;
  void* x = c.matrix(v[0], M, K, ldx);
  void* codes = c.matrix(v[1], M, K, ldc);
  int64_t kb = blocks_of(K);
  void* scales = c.matrix(v[2], M, kb, lds);
  c.need(c.ok && type_of(v[0]) >= 0 && is(v[1], kE4m3) && is(v[2], at::kFloat));
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  return g_quant_f8(x, type_of(v[0]), ldx, static_cast<int32_t>(M), static_cast<int32_t>(K), static_cast<uint8_t*>(codes), ldc,
                    static_cast<float*>(scales), lds, st);
}

// norm(x, weight, out, residual, total, codes, scales, eps)
long norm(PyObject* const* v, Py_ssize_t) {
  Call c;
  int64_t M = -1, K = -1, ldx = 0;
  moe_norm_opts_t o = {};
  void* x = c.matrix(v[0], M, K, ldx);
  const at::Tensor* w = c.tensor(v[1]);
  c.need(c.ok && type_of(v[0]) >= 0 && w->dim() == 1 && w->size(0) == K && (K == 1 || w->stride(0) == 1) &&
         (is(v[1], at::kFloat) || type_of(v[1]) == type_of(v[0])));
  auto same = [&](PyObject* t, int64_t& ld) -> void* {
    if (t == Py_None || !c.ok) return nullptr;
    void* p = c.matrix(t, M, K, ld);
    c.need(c.ok && type_of(t) == type_of(v[0]));
    return p;
  };
  o.out_dev = same(v[2], o.ldo);
  o.residual_dev = same(v[3], o.ldr);
  o.total_dev = same(v[4], o.ldt);
  c.need((v[5] == Py_None) == (v[6] == Py_None) && !(v[2] == Py_None && v[5] == Py_None));
  if (c.ok && v[5] != Py_None) {
    o.codes_dev = c.matrix(v[5], M, K, o.ldc);
    if (c.ok) o.codes = is(v[5], at::kChar) ? MOE_CODES_I8 : is(v[5], kE4m3) ? MOE_CODES_E4M3 : MOE_CODES_NONE;
    c.need(c.ok && o.codes != MOE_CODES_NONE);
    if (o.codes == MOE_CODES_I8) {
      o.scales_dev = c.vector(v[6], M);
    } else if (c.ok) {
      int64_t kb = blocks_of(K);
      o.scales_dev = static_cast<float*>(c.matrix(v[6], M, kb, o.lds));
      c.need(c.ok && is(v[6], at::kFloat));
    }
  }
  o.eps = PyFloat_AsDouble(v[7]);
  c.need(o.eps >= 0.0 && std::isfinite(o.eps));
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  return g_norm(x, type_of(v[0]), ldx, static_cast<int32_t>(M), static_cast<int32_t>(K), w->data_ptr(), type_of(v[1]), &o, st);
}

// linear_f8(a, a_scales, w, w_scales, out, act, bias, add[, exact])
long linear_f8(PyObject* const* v, Py_ssize_t n) {
  Call c;
  int64_t M = -1, K = -1, N = -1, lda = 0, ldw = 0, ldo = 0, ldsa = 0;
  const long act = PyLong_AsLong(v[5]);
  void* a = c.matrix(v[0], M, K, lda);
  void* w = c.matrix(v[2], N, K, ldw);
  c.need((act == 0 || act == 1) && !(act == 1 && N % 2));
  int64_t cols = act == 1 ? N / 2 : N, kb = blocks_of(K);
  void* out = c.matrix(v[4], M, cols, ldo);
  void* sa = c.matrix(v[1], M, kb, ldsa);
  const float* sw = c.blocks(v[3], -1, act == 1 ? 2 * blocks_of(cols) : blocks_of(cols), kb);
  const int exact = n > 8 ? PyObject_IsTrue(v[8]) : 0;
  c.need(c.ok && is(v[0], kE4m3) && is(v[2], kE4m3) && is(v[1], at::kFloat) && type_of(v[4]) >= 0 && exact >= 0);
  moe_linear_opts_t o = {static_cast<int32_t>(act), exact, nullptr, nullptr, 0};
  if (v[6] != Py_None) o.bias_dev = c.vector(v[6], N);
  if (v[7] != Py_None) {
    o.add_dev = c.matrix(v[7], M, cols, o.ldadd);
    c.need(c.ok && type_of(v[7]) == type_of(v[4]));
  }
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  return g_linear_f8(static_cast<const uint8_t*>(a), lda, static_cast<const float*>(sa), ldsa, static_cast<const uint8_t*>(w),
                     ldw, sw, static_cast<int32_t>(M), static_cast<int32_t>(N), static_cast<int32_t>(K), &o, out,
                     type_of(v[4]), ldo, st);
}

// lists(ids, offsets, pairs, ws)
long lists(PyObject* const* v, Py_ssize_t) {
  Call c;
  int64_t B = -1, K = -1, ld = 0, E1 = -1;
  void* ids = c.matrix(v[0], B, K, ld);
  c.need(c.ok && ld == K && is(v[0], at::kInt));
  int64_t R = B * K;
  int32_t* offsets = c.list(v[1], E1);
  int32_t* pairs = c.list(v[2], R);
  c.need(E1 >= 2 && E1 <= INT32_MAX);
  void* ws = nullptr;
  size_t bytes = 0;
  if (c.ok && v[3] != Py_None) {
    const at::Tensor* t = c.tensor(v[3]);
    c.need(c.ok && t->is_contiguous());
    if (c.ok && t->numel()) {
      ws = t->data_ptr();
      bytes = t->nbytes();
    }
  }
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  return g_lists(static_cast<const int32_t*>(ids), R, static_cast<int32_t>(E1 - 1), offsets, pairs, ws, bytes, st);
}

// grouped_f8(a, a_scales, w, w_scales, offsets, out, act, pairs, gather, scatter[, exact])
long grouped_f8(PyObject* const* v, Py_ssize_t n) {
  Call c;
  int64_t A = -1, O = -1, lda = 0, ldo = 0, ldsa = 0;
  const long act = PyLong_AsLong(v[6]), gather = PyLong_AsLong(v[8]);
  const int scatter = PyObject_IsTrue(v[9]), exact = n > 10 ? PyObject_IsTrue(v[10]) : 0;
  const at::Tensor* w = c.tensor(v[2]);
  if (!c.ok || w->dim() != 3 || w->scalar_type() != kE4m3) return kNotTaken;
  int64_t E = w->size(0), N = w->size(1), K = w->size(2), E1 = E + 1;
  const int64_t ldw = N == 1 ? K : w->stride(1), ldwe = E == 1 ? ((N - 1) * ldw + K + 15) & ~15LL : w->stride(0);
  c.need((w->stride(2) == 1 || K == 1) && ldw >= K && ldwe >= (N - 1) * ldw + K && E <= INT32_MAX && N <= INT32_MAX &&
         K <= INT32_MAX && (act == 0 || act == 1) && !(act == 1 && N % 2) && gather >= 0 && gather <= INT32_MAX && scatter >= 0 && exact >= 0);
  int64_t cols = act == 1 ? N / 2 : N, kb = blocks_of(K), R = -1;
  void* a = c.matrix(v[0], A, K, lda);
  void* sa = c.matrix(v[1], A, kb, ldsa);
  const float* sw = c.blocks(v[3], E, act == 1 ? 2 * blocks_of(cols) : blocks_of(cols), kb);
  int32_t* offsets = c.list(v[4], E1);
  void* out = c.matrix(v[5], O, cols, ldo);
  c.need(c.ok && is(v[0], kE4m3) && is(v[1], at::kFloat) && type_of(v[5]) >= 0);
  c.need((v[7] != Py_None) == (gather > 0 || scatter > 0));
  moe_grouped_opts_t o = {static_cast<int32_t>(act), static_cast<int32_t>(gather), scatter, exact, nullptr};
  if (c.ok && v[7] != Py_None) o.pairs_dev = c.list(v[7], R);
  else R = A < O ? A : O;
  void* st = c.stream();
  if (!c.ok) return kNotTaken;
  return g_grouped_f8(static_cast<const uint8_t*>(a), lda, static_cast<const float*>(sa), ldsa, A,
                      static_cast<const uint8_t*>(w->data_ptr()), ldw, ldwe, sw, offsets, R, static_cast<int32_t>(E),
                      static_cast<int32_t>(N), static_cast<int32_t>(K), &o, out, type_of(v[5]), ldo, O, st);
}

// No exception leaves: a tensor without storage, say, is one that _lib.py has to explain.  (The library throws none,
// so one means that it was not called.)
template <long (*F)(PyObject* const*, Py_ssize_t), int ARGS, int MORE = 0>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  long r = kNotTaken;
  try {
    if (n >= ARGS && n <= ARGS + MORE && g_linear && g_grouped_f8) r = F(args, n);
  } catch (...) {
    r = kNotTaken;
  }
  PyErr_Clear();
  return PyLong_FromLong(r);
}

// bind(gate, route, quant, linear, current raw stream, current device): four addresses, two callables
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[4];
  PyObject *stream, *device;
  if (!PyArg_ParseTuple(args, "KKKKOO", &f[0], &f[1], &f[2], &f[3], &stream, &device)) return nullptr;
  g_gate = reinterpret_cast<decltype(g_gate)>(f[0]);
  g_route = reinterpret_cast<decltype(g_route)>(f[1]);
  g_quant = reinterpret_cast<decltype(g_quant)>(f[2]);
  g_linear = reinterpret_cast<decltype(g_linear)>(f[3]);
  Py_INCREF(stream);
  Py_INCREF(device);
  g_raw_stream = stream;
  g_device = device;
  Py_RETURN_NONE;
}

// bind_f8(norm, quant_f8, linear_f8, lists, grouped_f8): five addresses
PyObject* bind_f8(PyObject*, PyObject* args) {
  unsigned long long f[5];
  if (!PyArg_ParseTuple(args, "KKKKK", &f[0], &f[1], &f[2], &f[3], &f[4])) return nullptr;
  g_norm = reinterpret_cast<decltype(g_norm)>(f[0]);
  g_quant_f8 = reinterpret_cast<decltype(g_quant_f8)>(f[1]);
  g_linear_f8 = reinterpret_cast<decltype(g_linear_f8)>(f[2]);
  g_lists = reinterpret_cast<decltype(g_lists)>(f[3]);
  g_grouped_f8 = reinterpret_cast<decltype(g_grouped_f8)>(f[4]);
  Py_RETURN_NONE;
}

#define FAST(F) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"gate", FAST((entry<gate, 5, 1>))},
                         {"route", FAST((entry<route, 10>))},
                         {"quant", FAST((entry<quant, 3>))},
                         {"linear", FAST((entry<linear, 8>))},
                         {"norm", FAST((entry<norm, 8>))},
                         {"quant_f8", FAST((entry<quant_f8, 3>))},
                         {"linear_f8", FAST((entry<linear_f8, 8, 1>))},
                         {"lists", FAST((entry<lists, 4>))},
                         {"grouped_f8", FAST((entry<grouped_f8, 10, 1>))},
                         {"bind", bind, METH_VARARGS, nullptr},
                         {"bind_f8", bind_f8, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dense() { return PyModule_Create(&module); }
