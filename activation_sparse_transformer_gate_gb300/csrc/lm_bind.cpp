// lm_bind.cpp -- argument marshalling of the operators around the FFN for
// Python (module _lm): tensors are checked and their addresses handed to the
// C entry points of include/twell_lm.h.
//
// A decoded token's calls last a few microseconds on the GPU, as long as it
// takes Python to ask eight tensors for their type, size, place and address
// and ctypes to convert fifteen arguments (6 us a call so); here that is about
// half a microsecond.
//
// Every function takes its arguments by position and returns the status code.
// A tensor argument may be None (NULL) or an integer (a raw device pointer).
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAStream.h>

#include "twell_lm.h"

namespace {

// The arguments of one call, taken in order.  The first failure is kept; what
// follows it is not looked at.
class Args {
 public:
  Args(PyObject *const *a, Py_ssize_t n) : a_(a), n_(n) {}

  PyObject *next() {
    if (at_ >= n_) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "too few arguments");
      return nullptr;
    }
    return a_[at_++];
  }
  long long integer() {
    PyObject *o = failed() ? nullptr : next();
    return o ? PyLong_AsLongLong(o) : 0;
  }
  int small() {
    const long long v = integer();
    if (v > INT32_MAX || v < INT32_MIN) fail(TWELL_ERR_ARG);
    return (int)v;
  }
  float real() {
    PyObject *o = failed() ? nullptr : next();
    return o ? (float)PyFloat_AsDouble(o) : 0.f;
  }
  // An operand of `count` elements.
  void *tensor(at::ScalarType type, long long count) {
    PyObject *o = failed() ? nullptr : next();
    void *p = nullptr;
    if (!o || raw(o, &p)) return p;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != type) return fail(TWELL_ERR_DTYPE);
    if (t.numel() != count || !t.is_cuda() || !t.is_contiguous()) return fail(TWELL_ERR_ARG);
    return t.data_ptr();
  }
  // A [rows][cols] operand with a row pitch (elements).
  void *pitched(at::ScalarType type, long long rows, long long cols, long long pitch) {
    PyObject *o = failed() ? nullptr : next();
    void *p = nullptr;
    if (!o || raw(o, &p)) return p;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != type) return fail(TWELL_ERR_DTYPE);
    if (!t.is_cuda() || t.dim() != 2 || t.size(0) != rows ||
        (t.size(1) != cols && t.size(1) != pitch) || (t.size(1) > 1 && t.stride(1) != 1) ||
        (rows > 1 && t.stride(0) != pitch))
      return fail(TWELL_ERR_ARG);
    return t.data_ptr();
  }
  // Token ids: int32 or int64 (a raw pointer: int32).
  void *tokens(long long count, int *bytes) {
    *bytes = 4;
    PyObject *o = failed() ? nullptr : next();
    void *p = nullptr;
    if (!o || raw(o, &p)) return p;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() == at::kLong) *bytes = 8;
    else if (t.scalar_type() != at::kInt) return fail(TWELL_ERR_DTYPE);
    if (t.numel() != count || !t.is_cuda() || !t.is_contiguous()) return fail(TWELL_ERR_ARG);
    return t.data_ptr();
  }
  // Scratch of at least the bytes that the next argument states.
  void *scratch(size_t *bytes) {
    PyObject *o = failed() ? nullptr : next();
    const long long n = integer();
    *bytes = n < 0 ? 0 : (size_t)n;
    void *p = nullptr;
    if (!o || failed() || raw(o, &p)) return p;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || (long long)t.nbytes() < n) return fail(TWELL_ERR_WORKSPACE);
    return t.data_ptr();
  }
  // Element type of the twell_dtype that the call states.
  at::ScalarType type(int dtype) {
    if (dtype != TWELL_F32 && dtype != TWELL_BF16) fail(TWELL_ERR_DTYPE);
    return dtype == TWELL_BF16 ? at::kBFloat16 : at::kFloat;
  }
  // The last argument: None for the current stream, a raw handle, or a stream.
  void *stream() {
    PyObject *o = failed() ? nullptr : next();
    if (!o) return nullptr;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    void *p = h ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(h);
    return p;
  }
  void *fail(int code) {
    if (!code_) code_ = code;
    return nullptr;
  }
  bool failed() const { return code_ != 0 || PyErr_Occurred(); }
  int code() const { return code_; }

  // Peeks at a later argument (sizes stand behind the tensors they describe).
  // (What is not a number raises where its turn comes.)
  long long ahead(Py_ssize_t i) const {
    const long long v = i < n_ ? PyLong_AsLongLong(a_[i]) : 0;
    if (!PyErr_Occurred()) return v;
    PyErr_Clear();
    return 0;
  }

 private:
  bool raw(PyObject *o, void **p) {
    if (o == Py_None) return true;
    if (PyLong_Check(o)) {
      *p = PyLong_AsVoidPtr(o);
      return true;
    }
    if (THPVariable_Check(o)) return false;
    PyErr_SetString(PyExc_TypeError, "a tensor, a device pointer or None is wanted");
    return true;
  }

  PyObject *const *a_;
  Py_ssize_t n_, at_ = 0;
  int code_ = 0;
};

// Runs `call` unless an argument failed.
template <typename F>
PyObject *finish(const Args &a, F call) {
  if (PyErr_Occurred()) return nullptr;
  return PyLong_FromLong(a.code() ? a.code() : (long)call());
}

constexpr at::ScalarType F32 = at::kFloat, I8 = at::kChar, I32 = at::kInt;

// tokens, table, T, V, D, dtype, scale, pad_id, out, status, stream
PyObject *embed_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long T = a.ahead(2), V = a.ahead(3), D = a.ahead(4);
  const at::ScalarType t = a.type((int)a.ahead(5));
  int bytes;
  const void *tok = a.tokens(T, &bytes), *table = a.tensor(t, V * D);
  const int iT = a.small(), iV = a.small(), iD = a.small(), dt = a.small();
  const float scale = a.real();
  const long long pad = a.integer();
  void *out = a.tensor(t, T * D), *st = a.tensor(I32, 1), *s = a.stream();
  return finish(a, [&] {
    return twell_embed_forward(tok, bytes, table, iT, iV, iD, dt, scale, pad, out, (int32_t *)st, s);
  });
}

// tokens, dy, T, V, D, dtype, scale, pad_id, dtable, status, workspace, bytes, stream
PyObject *embed_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long T = a.ahead(2), V = a.ahead(3), D = a.ahead(4);
  const at::ScalarType t = a.type((int)a.ahead(5));
  int bytes;
  size_t nws;
  const void *tok = a.tokens(T, &bytes), *dy = a.tensor(t, T * D);
  const int iT = a.small(), iV = a.small(), iD = a.small(), dt = a.small();
  const float scale = a.real();
  const long long pad = a.integer();
  void *dtable = a.tensor(F32, V * D), *st = a.tensor(I32, 1), *ws = a.scratch(&nws);
  void *s = a.stream();
  return finish(a, [&] {
    return twell_embed_backward(tok, bytes, dy, iT, iV, iD, dt, scale, pad, (float *)dtable,
                                (int32_t *)st, ws, nws, s);
  });
}

// x, residual, weight, T, D, dtype, eps, s, y, q, qscale, rstd, stream
PyObject *add_rmsnorm_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long T = a.ahead(3), D = a.ahead(4);
  const at::ScalarType t = a.type((int)a.ahead(5));
  const void *x = a.tensor(t, T * D), *res = a.tensor(t, T * D), *w = a.tensor(F32, D);
  const int iT = a.small(), iD = a.small(), dt = a.small();
  const float eps = a.real();
  void *s = a.tensor(t, T * D), *y = a.tensor(t, T * D), *q = a.tensor(I8, T * D);
  void *qs = a.tensor(F32, T), *rstd = a.tensor(F32, T), *st = a.stream();
  return finish(a, [&] {
    return twell_add_rmsnorm_forward(x, res, (const float *)w, iT, iD, dt, eps, s, y, (int8_t *)q,
                                     (float *)qs, (float *)rstd, st);
  });
}

// s, weight, rstd, dy, ds, T, D, dtype, dx, dweight, workspace, bytes, stream
PyObject *add_rmsnorm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long T = a.ahead(5), D = a.ahead(6);
  const at::ScalarType t = a.type((int)a.ahead(7));
  size_t nws;
  const void *s = a.tensor(t, T * D), *w = a.tensor(F32, D), *rstd = a.tensor(F32, T);
  const void *dy = a.tensor(t, T * D), *ds = a.tensor(t, T * D);
  const int iT = a.small(), iD = a.small(), dt = a.small();
  void *dx = a.tensor(t, T * D), *dw = a.tensor(F32, D), *ws = a.scratch(&nws), *st = a.stream();
  return finish(a, [&] {
    return twell_add_rmsnorm_backward(s, (const float *)w, (const float *)rstd, dy, ds, iT, iD, dt,
                                      dx, (float *)dw, ws, nws, st);
  });
}

// a, rows, cols, dtype, q, scale, stream
PyObject *q8_quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long R = a.ahead(1), C = a.ahead(2);
  const void *m = a.tensor(a.type((int)a.ahead(3)), R * C);
  const int rows = a.small(), cols = a.small(), dt = a.small();
  void *q = a.tensor(I8, R * C), *scale = a.tensor(F32, R), *s = a.stream();
  return finish(a, [&] {
    return twell_q8_quantize(m, rows, cols, dt, (int8_t *)q, (float *)scale, s);
  });
}

// aq, ascale, wq, wscale, bias, M, N, K, dtype, y, status, workspace, bytes, stream
PyObject *q8_matmul(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long M = a.ahead(5), N = a.ahead(6), K = a.ahead(7);
  const at::ScalarType t = a.type((int)a.ahead(8));
  size_t nws;
  const void *aq = a.tensor(I8, M * K), *sa = a.tensor(F32, M), *wq = a.tensor(I8, N * K);
  const void *sw = a.tensor(F32, N), *bias = a.tensor(F32, N);
  const int iM = a.small(), iN = a.small(), iK = a.small(), dt = a.small();
  void *y = a.tensor(t, M * N), *st = a.tensor(I32, 1), *ws = a.scratch(&nws), *s = a.stream();
  return finish(a, [&] {
    return twell_q8_matmul((const int8_t *)aq, (const float *)sa, (const int8_t *)wq,
                           (const float *)sw, (const float *)bias, iM, iN, iK, dt, y, (int32_t *)st,
                           ws, nws, s);
  });
}

// z, ldz, ids, teacher, row_weight, T, V, k, dtype, tau, loss, stats, dz, status, stream
PyObject *distill_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long L = a.ahead(1), T = a.ahead(5), V = a.ahead(6), k = a.ahead(7);
  const at::ScalarType t = a.type((int)a.ahead(8));
  const void *z = a.pitched(t, T, V, L);
  const long long ldz = a.integer();
  const void *ids = a.tensor(I32, T * k), *te = a.tensor(F32, T * k), *w = a.tensor(F32, T);
  const int iT = a.small(), iV = a.small(), ik = a.small(), dt = a.small();
  const float tau = a.real();
  void *loss = a.tensor(F32, T), *stats = a.tensor(F32, 2 * T), *dz = a.pitched(t, T, V, L);
  void *st = a.tensor(I32, 1), *s = a.stream();
  return finish(a, [&] {
    return twell_distill_forward(z, ldz, (const int32_t *)ids, (const float *)te, (const float *)w,
                                 iT, iV, ik, dt, tau, (float *)loss, (float *)stats, dz,
                                 (int32_t *)st, s);
  });
}

// z, ldz, ids, teacher, stats, row_grad, T, V, k, dtype, tau, dz, status, stream
PyObject *distill_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long L = a.ahead(1), T = a.ahead(6), V = a.ahead(7), k = a.ahead(8);
  const at::ScalarType t = a.type((int)a.ahead(9));
  const void *z = a.pitched(t, T, V, L);
  const long long ldz = a.integer();
  const void *ids = a.tensor(I32, T * k), *te = a.tensor(F32, T * k);
  const void *stats = a.tensor(F32, 2 * T), *g = a.tensor(F32, T);
  const int iT = a.small(), iV = a.small(), ik = a.small(), dt = a.small();
  const float tau = a.real();
  void *dz = a.pitched(t, T, V, L), *st = a.tensor(I32, 1), *s = a.stream();
  return finish(a, [&] {
    return twell_distill_backward(z, ldz, (const int32_t *)ids, (const float *)te,
                                  (const float *)stats, (const float *)g, iT, iV, ik, dt, tau, dz,
                                  (int32_t *)st, s);
  });
}

using Method = PyObject *(PyObject *, PyObject *const *, Py_ssize_t);

// No C++ exception leaves through Python's C frames.
template <Method *F>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define TWELL_METHOD(name) \
  {#name, (PyCFunction)(void (*)(void))guarded<name>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    TWELL_METHOD(embed_forward),       TWELL_METHOD(embed_backward),
    TWELL_METHOD(add_rmsnorm_forward), TWELL_METHOD(add_rmsnorm_backward),
    TWELL_METHOD(q8_quantize),         TWELL_METHOD(q8_matmul),
    TWELL_METHOD(distill_forward),     TWELL_METHOD(distill_backward),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm",
                      "Argument marshalling of the operators around the FFN.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm(void) { return PyModule_Create(&module); }
