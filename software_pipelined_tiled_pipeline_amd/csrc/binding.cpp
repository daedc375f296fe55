// The short way through the Python binding of the fused operators.
//
// A call of a few microseconds on the GPU should not spend twice that in
// Python: these functions check a call's tensors, allocate its outputs and call
// the library, and return None for whatever is not plainly right, which
// fused.py then looks at for itself, to refuse it with a reason or to register
// a workspace.  Each takes the library function's address, the current device
// and stream, the operand type (0 f16, 1 bf16) and the call's own arguments.
// Nothing is computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pgemm.h"

namespace {

using at::ScalarType;

constexpr ScalarType kTypes[2] = {at::kHalf, at::kBFloat16};
constexpr int kFixed = 4;  // address, device, stream, type

struct Call {
  PyObject *const *args;
  void *entry;
  int64_t dev;
  void *stream;
  ScalarType type;
  bool ok = true;

  Call(PyObject *const *a, Py_ssize_t n, Py_ssize_t own) : args(a + kFixed) {
    if (n != kFixed + own) {
      ok = false;
      return;
    }
    entry = PyLong_AsVoidPtr(a[0]);
    dev = PyLong_AsLongLong(a[1]);
    stream = PyLong_AsVoidPtr(a[2]);
    const long long t = PyLong_AsLongLong(a[3]);
    type = kTypes[t == 1];
    if (PyErr_Occurred() || !entry) ok = false;
  }
  // Argument i as a contiguous tensor of a type on the current device, with
  // the given sizes (-1: any); null, and the call is not ok, if it is not.
  const at::Tensor *tensor(int i, ScalarType st, std::initializer_list<int64_t> sizes) {
    if (!ok || !THPVariable_Check(args[i])) return fail();
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    if (t.scalar_type() != st || !t.is_cuda() || t.get_device() != dev || t.dim() != (int64_t)sizes.size()) return fail();
    int64_t d = 0;
    for (const int64_t want : sizes) {
      if (want >= 0 && t.size(d) != want) return fail();
      ++d;
    }
    return t.is_contiguous() ? &t : fail();
  }
  const at::Tensor *fail() {
    ok = false;
    return nullptr;
  }
  int64_t integer(int i) {
    const long long v = ok ? PyLong_AsLongLong(args[i]) : 0;
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  bool truth(int i) {
    const int v = ok ? PyObject_IsTrue(args[i]) : 0;
    if (v < 0) ok = false;
    return v > 0;
  }
  bool none(int i) const { return args[i] == Py_None; }
};

template <typename U = uint16_t>
U *ptr(const at::Tensor *t) {
  return t ? static_cast<U *>(t->data_ptr()) : nullptr;
}
at::Tensor made(const at::Tensor *like, ScalarType st, at::IntArrayRef sizes) {
  return at::empty(sizes, like->options().dtype(st).requires_grad(false));
}

PyObject *nothing() {
  PyErr_Clear();
  Py_RETURN_NONE;
}
PyObject *pair(at::Tensor a, at::Tensor b) {
  PyObject *t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(a)));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(b)));
  return t;
}

// A C++ exception (out of memory) is left to fused.py, which meets it again.
template <typename F>
PyObject *guarded(F &&f) {
  try {
    return f();
  } catch (...) {
    return nothing();
  }
}

int64_t per(int64_t a, int64_t b) { return (a + b - 1) / b; }

// x, w, act, save
PyObject *gated(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, 4);
    const at::Tensor *x = c.ok ? c.tensor(0, c.type, {-1, -1}) : nullptr;
    const at::Tensor *w = x ? c.tensor(1, c.type, {-1, x->size(1)}) : nullptr;
    const int act = (int)c.integer(2);
    const bool save = c.truth(3);
    if (!c.ok || w->size(0) % 2) return nothing();
    const int64_t M = x->size(0), F = w->size(0) / 2, D = x->size(1);
    at::Tensor h = made(x, c.type, {M, F}), saved;
    if (save) saved = made(x, at::kFloat, {M, per(F, 4), 8});
    const auto f = reinterpret_cast<decltype(&pgemm_f16_gated)>(c.entry);
    if (f(ptr(x), ptr(w), ptr(&h), save ? ptr<float>(&saved) : nullptr, M, F, D, act, c.stream) != PGEMM_OK) return nothing();
    return save ? pair(std::move(h), std::move(saved)) : THPVariable_Wrap(std::move(h));
  });
}

// dh, x, w, saved or None, act
PyObject *gated_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, 5);
    const at::Tensor *x = c.ok ? c.tensor(1, c.type, {-1, -1}) : nullptr;
    const at::Tensor *w = x ? c.tensor(2, c.type, {-1, x->size(1)}) : nullptr;
    if (!w || w->size(0) % 2) return nothing();
    const int64_t M = x->size(0), F = w->size(0) / 2, D = x->size(1);
    const at::Tensor *dh = c.tensor(0, c.type, {M, F});
    const at::Tensor *saved = dh && !c.none(3) ? c.tensor(3, at::kFloat, {M, per(F, 4), 8}) : nullptr;
    const int act = (int)c.integer(4);
    if (!c.ok) return nothing();
    at::Tensor dx = made(x, c.type, {M, D}), dw = made(x, c.type, {2 * F, D});
    const auto f = reinterpret_cast<decltype(&pgemm_f16_gated_bwd)>(c.entry);
    if (f(ptr(dh), ptr(x), ptr(w), ptr<float>(saved), ptr(&dx), ptr(&dw), M, F, D, act, c.stream) != PGEMM_OK)
      return nothing();
    return pair(std::move(dx), std::move(dw));
  });
}

// x, w, target, ignore_index
PyObject *xent(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, 4);
    const at::Tensor *x = c.ok ? c.tensor(0, c.type, {-1, -1}) : nullptr;
    const at::Tensor *w = x ? c.tensor(1, c.type, {-1, x->size(1)}) : nullptr;
    const at::Tensor *target = w ? c.tensor(2, at::kLong, {x->size(0)}) : nullptr;
    const int64_t ignore = c.integer(3);
    if (!c.ok) return nothing();
    const int64_t M = x->size(0), V = w->size(0), D = x->size(1);
    at::Tensor loss = made(x, at::kFloat, {M}), lse = made(x, at::kFloat, {M});
    const auto f = reinterpret_cast<decltype(&pgemm_f16_xent)>(c.entry);
    if (f(ptr(x), ptr(w), ptr<int64_t>(target), ptr<float>(&loss), ptr<float>(&lse), M, V, D, ignore, c.stream) != PGEMM_OK)
      return nothing();
    return pair(std::move(loss), std::move(lse));
  });
}

// dloss, x, w, target, lse, ignore_index
PyObject *xent_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, 6);
    const at::Tensor *x = c.ok ? c.tensor(1, c.type, {-1, -1}) : nullptr;
    const at::Tensor *w = x ? c.tensor(2, c.type, {-1, x->size(1)}) : nullptr;
    const at::Tensor *target = w ? c.tensor(3, at::kLong, {x->size(0)}) : nullptr;
    const at::Tensor *lse = target ? c.tensor(4, at::kFloat, {x->size(0)}) : nullptr;
    const at::Tensor *dloss = lse ? c.tensor(0, at::kFloat, {x->size(0)}) : nullptr;
    const int64_t ignore = c.integer(5);
    if (!c.ok) return nothing();
    const int64_t M = x->size(0), V = w->size(0), D = x->size(1);
    at::Tensor dx = made(x, c.type, {M, D}), dw = made(x, c.type, {V, D});
    const auto f = reinterpret_cast<decltype(&pgemm_f16_xent_bwd)>(c.entry);
    if (f(ptr<float>(dloss), 1, ptr(x), ptr(w), ptr<int64_t>(target), ptr<float>(lse), ptr(&dx), ptr(&dw), M, V, D, ignore,
          c.stream) != PGEMM_OK)
      return nothing();
    return pair(std::move(dx), std::move(dw));
  });
}

// x, q, scale, zero or None, group, and for the gated block act
PyObject *q4_call(PyObject *const *args, Py_ssize_t n, bool block) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, block ? 6 : 5);
    const at::Tensor *x = c.ok ? c.tensor(0, c.type, {-1, -1}) : nullptr;
    const int64_t group = c.integer(4);
    const int act = block ? (int)c.integer(5) : 0;
    if (!c.ok || group <= 0) return nothing();
    const int64_t M = x->size(0), K = x->size(1), groups = per(K, group);
    const at::Tensor *q = c.tensor(1, at::kByte, {-1, per(K, 32) * 16});
    const at::Tensor *scale = q ? c.tensor(2, c.type, {q->size(0), groups}) : nullptr;
    const at::Tensor *zero = scale && !c.none(3) ? c.tensor(3, at::kByte, {q->size(0), groups}) : nullptr;
    if (!c.ok || (block && q->size(0) % 2)) return nothing();
    const int64_t N = block ? q->size(0) / 2 : q->size(0);
    at::Tensor out = made(x, c.type, {M, N});
    pgemm_status st;
    if (block)
      st = reinterpret_cast<decltype(&pgemm_f16_q4_gated)>(c.entry)(ptr(x), ptr<uint8_t>(q), ptr(scale), ptr<uint8_t>(zero),
                                                                    ptr(&out), M, N, K, group, act, c.stream);
    else
      st = reinterpret_cast<decltype(&pgemm_f16_q4)>(c.entry)(ptr(x), ptr<uint8_t>(q), ptr(scale), ptr<uint8_t>(zero),
                                                              ptr(&out), M, N, K, group, c.stream);
    return st == PGEMM_OK ? THPVariable_Wrap(std::move(out)) : nothing();
  });
}
PyObject *q4(PyObject *, PyObject *const *args, Py_ssize_t n) { return q4_call(args, n, false); }
PyObject *q4_gated(PyObject *, PyObject *const *args, Py_ssize_t n) { return q4_call(args, n, true); }

#define METHOD(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(gated),  METHOD(gated_bwd), METHOD(xent),      METHOD(xent_bwd),
                         METHOD(q4),     METHOD(q4_gated),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
