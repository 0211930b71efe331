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

#include <memory>
#include <vector>

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

// x, gate, ld, bias, starts, B, h0, T, D, dtype, h, hT, states, status, stream
PyObject *recur_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long L = a.ahead(2), B = a.ahead(5), T = a.ahead(7), D = a.ahead(8);
  const at::ScalarType t = a.type((int)a.ahead(9));
  const void *x = a.pitched(t, T, D, L), *gate = a.pitched(t, T, D, L);
  const long long ld = a.integer();
  const void *bias = a.tensor(F32, D), *starts = a.tensor(I32, B + 1);
  const int iB = a.small();
  const void *h0 = a.tensor(F32, B * D);
  const int iT = a.small(), iD = a.small(), dt = a.small();
  void *h = a.tensor(t, T * D), *hT = a.tensor(F32, B * D);
  void *states = a.tensor(F32, twell_recur_states((int)T) * D), *st = a.tensor(I32, 1);
  void *s = a.stream();
  return finish(a, [&] {
    return twell_recur_forward(x, gate, ld, (const float *)bias, (const int32_t *)starts, iB,
                               (const float *)h0, iT, iD, dt, h, (float *)hT, (float *)states,
                               (int32_t *)st, s);
  });
}

// x, gate, ld, bias, starts, B, h0, states, dh, dhT, T, D, dtype, dx, dgate, dbias, dh0, status,
// stream
PyObject *recur_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long L = a.ahead(2), B = a.ahead(5), T = a.ahead(10), D = a.ahead(11);
  const at::ScalarType t = a.type((int)a.ahead(12));
  const void *x = a.pitched(t, T, D, L), *gate = a.pitched(t, T, D, L);
  const long long ld = a.integer();
  const void *bias = a.tensor(F32, D), *starts = a.tensor(I32, B + 1);
  const int iB = a.small();
  const void *h0 = a.tensor(F32, B * D);
  const void *states = a.tensor(F32, twell_recur_states((int)T) * D);
  const void *dh = a.tensor(t, T * D), *dhT = a.tensor(F32, B * D);
  const int iT = a.small(), iD = a.small(), dt = a.small();
  void *dx = a.pitched(t, T, D, L), *dgate = a.pitched(t, T, D, L);
  void *dbias = a.tensor(F32, D), *dh0 = a.tensor(F32, B * D), *st = a.tensor(I32, 1);
  void *s = a.stream();
  return finish(a, [&] {
    return twell_recur_backward(x, gate, ld, (const float *)bias, (const int32_t *)starts, iB,
                                (const float *)h0, (const float *)states, dh, (const float *)dhT,
                                iT, iD, dt, dx, dgate, (float *)dbias, (float *)dh0, (int32_t *)st,
                                s);
  });
}

// z, ldz, tokens, old_logp, ref_logp, advantage, row_weight, T, V, dtype, tau, clip_low, clip_high,
// beta, loss, logp, stats, dz, status, stream
PyObject *policy_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long L = a.ahead(1), T = a.ahead(7), V = a.ahead(8);
  const at::ScalarType t = a.type((int)a.ahead(9));
  int bytes;
  const void *z = a.pitched(t, T, V, L);
  const long long ldz = a.integer();
  const void *tok = a.tokens(T, &bytes), *old = a.tensor(F32, T), *ref = a.tensor(F32, T);
  const void *adv = a.tensor(F32, T), *w = a.tensor(F32, T);
  const int iT = a.small(), iV = a.small(), dt = a.small();
  const float tau = a.real(), low = a.real(), high = a.real(), beta = a.real();
  void *loss = a.tensor(F32, T), *logp = a.tensor(F32, T), *stats = a.tensor(F32, 2 * T);
  void *dz = a.pitched(t, T, V, L), *st = a.tensor(I32, 1), *s = a.stream();
  return finish(a, [&] {
    return twell_policy_forward(z, ldz, tok, bytes, (const float *)old, (const float *)ref,
                                (const float *)adv, (const float *)w, iT, iV, dt, tau, low, high,
                                beta, (float *)loss, (float *)logp, (float *)stats, dz,
                                (int32_t *)st, s);
  });
}

// z, ldz, tokens, old_logp, ref_logp, advantage, logp, stats, row_grad, T, V, dtype, tau, clip_low,
// clip_high, beta, dz, status, stream
PyObject *policy_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  const long long L = a.ahead(1), T = a.ahead(9), V = a.ahead(10);
  const at::ScalarType t = a.type((int)a.ahead(11));
  int bytes;
  const void *z = a.pitched(t, T, V, L);
  const long long ldz = a.integer();
  const void *tok = a.tokens(T, &bytes), *old = a.tensor(F32, T), *ref = a.tensor(F32, T);
  const void *adv = a.tensor(F32, T), *logp = a.tensor(F32, T), *stats = a.tensor(F32, 2 * T);
  const void *g = a.tensor(F32, T);
  const int iT = a.small(), iV = a.small(), dt = a.small();
  const float tau = a.real(), low = a.real(), high = a.real(), beta = a.real();
  void *dz = a.pitched(t, T, V, L), *st = a.tensor(I32, 1), *s = a.stream();
  return finish(a, [&] {
    return twell_policy_backward(z, ldz, tok, bytes, (const float *)old, (const float *)ref,
                                 (const float *)adv, (const float *)logp, (const float *)stats,
                                 (const float *)g, iT, iV, dt, tau, low, high, beta, dz,
                                 (int32_t *)st, s);
  });
}

// A tensor of an AdamW list as it was when its row was made.  `t` is what Python's object holds,
// not a copy of it, so that other memory given to it shows here.
struct Held {
  at::Tensor t;
  caffe2::TypeMeta type;
  int64_t n, offset;
  const void *memory;
};
constexpr const char *LIST = "twell_adamw_list";
using List = std::vector<Held>;

// Whether the tensors still are what the rows were made from: a row would keep what was freed.
// (70 tensors in under 0.1 us; by what Python's objects say, 0.6.)
int same_tensors(const List &list) {
  for (const Held &h : list) {
    const c10::TensorImpl *i = h.t.unsafeGetTensorImpl();
    if (i->dtype() != h.type) return TWELL_ERR_DTYPE;
    if (i->numel() != h.n || i->storage_offset() != h.offset || !i->is_contiguous() ||
        !i->has_storage() || i->unsafe_storage().data() != h.memory)
      return TWELL_ERR_ARG;
  }
  return TWELL_OK;
}

// tensors (a tuple, seven a row, None where the row has none), the rows (address of the host's
// array), count; the list, or None where a row is not what its tensors are
PyObject *adamw_list(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  PyObject *const tuple = a.next();
  const twell_adamw_tensor *rows = (const twell_adamw_tensor *)a.integer();
  const long long count = a.integer();
  if (PyErr_Occurred()) return nullptr;
  if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != 7 * count) {
    PyErr_SetString(PyExc_TypeError, "a tuple of seven tensors a row is wanted");
    return nullptr;
  }
  auto list = std::make_unique<List>();
  for (long long i = 0; i < 7 * count; ++i) {
    const twell_adamw_tensor &r = rows[i / 7];
    const void *const at[7] = {r.param, r.grad, r.m, r.v, r.mscale, r.vscale, r.copy};
    const int k = (int)(i % 7);
    PyObject *o = PyTuple_GET_ITEM(tuple, i);
    if (o != Py_None && !THPVariable_Check(o)) {
      PyErr_SetString(PyExc_TypeError, "a tensor or None is wanted");
      return nullptr;
    }
    if (o == Py_None) {
      if (at[k]) Py_RETURN_NONE;
      continue;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.const_data_ptr() != at[k] || t.numel() != (k == 4 || k == 5 ? (r.n + 255) / 256 : r.n))
      Py_RETURN_NONE;
    list->push_back(Held{t, t.dtype(), t.numel(), t.storage_offset(),
                         t.unsafeGetTensorImpl()->unsafe_storage().data()});
  }
  PyObject *c = PyCapsule_New(list.get(), LIST, [](PyObject *o) {
    delete (List *)PyCapsule_GetPointer(o, LIST);
  });
  if (c) list.release();
  return c;
}

// list, the rows made from its tensors (address of the host's array), count, grad_dtype, state_bits, lr, beta1, beta2, eps, step,
// seed, grad_scale, dynamic, stream
PyObject *adamw_step(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Args a(args, n);
  PyObject *const o = a.next();
  const List *const list = o ? (const List *)PyCapsule_GetPointer(o, LIST) : nullptr;
  const twell_adamw_tensor *rows = (const twell_adamw_tensor *)a.integer();
  const int count = a.small(), gt = a.small(), bits = a.small();
  const float lr = a.real(), b1 = a.real(), b2 = a.real(), eps = a.real();
  const long long step = a.integer(), seed = a.integer();
  const void *scale = a.tensor(F32, 1), *dyn = a.tensor(I32, 4);
  void *s = a.stream();
  if (!a.failed()) {
    const int st = same_tensors(*list);
    if (st != TWELL_OK) a.fail(st);
  }
  return finish(a, [&] {
    return twell_adamw_step(rows, count, gt, bits, lr, b1, b2, eps, step,
                            (uint32_t)seed, (const float *)scale, (const twell_adamw_dynamic *)dyn,
                            s);
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
    TWELL_METHOD(recur_forward),       TWELL_METHOD(recur_backward),
    TWELL_METHOD(policy_forward),      TWELL_METHOD(policy_backward),
    TWELL_METHOD(adamw_list),          TWELL_METHOD(adamw_step),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm",
                      "Argument marshalling of the operators around the FFN.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm(void) { return PyModule_Create(&module); }
