// dense_binding.cpp -- the short way from Python to the dense side's entry points.
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

// No exception leaves: a tensor without storage, say, is one that _lib.py has to explain.  (The library throws none,
// so one means that it was not called.)
template <long (*F)(PyObject* const*, Py_ssize_t), int ARGS, int MORE = 0>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  long r = kNotTaken;
  try {
    if (n >= ARGS && n <= ARGS + MORE && g_linear) r = F(args, n);
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

#define FAST(F) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"gate", FAST((entry<gate, 5, 1>))},
                         {"route", FAST((entry<route, 10>))},
                         {"quant", FAST((entry<quant, 3>))},
                         {"linear", FAST((entry<linear, 8>))},
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dense() { return PyModule_Create(&module); }
