// The short way through the Python binding of the fused and serving operators.
//
// A call of a few microseconds on the GPU should not spend twice that in
// Python: these functions check a call's tensors, allocate its outputs and call
// the library, and return None for whatever is not plainly right, which
// fused.py (or serve.py) then looks at for itself, to refuse it with a reason or to register
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

// x
PyObject *quant_i8(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, 1);
    const at::Tensor *x = c.ok ? c.tensor(0, c.type, {-1, -1}) : nullptr;
    if (!c.ok) return nothing();
    const int64_t M = x->size(0), K = x->size(1);
    at::Tensor q = made(x, at::kChar, {M, per(K, 16) * 16}), scale = made(x, at::kFloat, {M});
    const auto f = reinterpret_cast<decltype(&pgemm_f16_quant_i8)>(c.entry);
    if (f(ptr(x), ptr<int8_t>(&q), ptr<float>(&scale), M, K, c.stream) != PGEMM_OK) return nothing();
    return pair(std::move(q), std::move(scale));
  });
}

// x, w, scale, xs or None, and for the gated block act
PyObject *i8_call(PyObject *const *args, Py_ssize_t n, bool block) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, block ? 5 : 4);
    const bool given = c.ok && !c.none(3);
    const at::Tensor *x = c.ok ? c.tensor(0, given ? at::kChar : c.type, {-1, -1}) : nullptr;
    const int act = block ? (int)c.integer(4) : 0;
    if (!c.ok) return nothing();
    const int64_t M = x->size(0), K = x->size(1);
    const at::Tensor *xs = given ? c.tensor(3, at::kFloat, {M}) : nullptr;
    const at::Tensor *w = c.tensor(1, at::kChar, {-1, per(K, 16) * 16});
    const at::Tensor *scale = w ? c.tensor(2, at::kFloat, {w->size(0)}) : nullptr;
    if (!c.ok || (given && K % 16) || (block && w->size(0) % 2) || (given && M == 0)) return nothing();
    const int64_t N = block ? w->size(0) / 2 : w->size(0);
    at::Tensor out = made(x, c.type, {M, N});
    pgemm_status st;
    if (block)
      st = reinterpret_cast<decltype(&pgemm_f16_i8_gated)>(c.entry)(x->data_ptr(), ptr<float>(xs), ptr<int8_t>(w), ptr<float>(scale),
                                                                    ptr(&out), M, N, K, act, c.stream);
    else
      st = reinterpret_cast<decltype(&pgemm_f16_i8)>(c.entry)(x->data_ptr(), ptr<float>(xs), ptr<int8_t>(w), ptr<float>(scale),
                                                              ptr(&out), M, N, K, c.stream);
    return st == PGEMM_OK ? THPVariable_Wrap(std::move(out)) : nothing();
  });
}
PyObject *i8(PyObject *, PyObject *const *args, Py_ssize_t n) { return i8_call(args, n, false); }
PyObject *i8_gated(PyObject *, PyObject *const *args, Py_ssize_t n) { return i8_call(args, n, true); }

// x, router, w, down, top_k, normalize, act, routing
PyObject *moe(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, 8);
    const at::Tensor *x = c.ok ? c.tensor(0, c.type, {-1, -1}) : nullptr;
    const at::Tensor *router = x ? c.tensor(1, c.type, {-1, x->size(1)}) : nullptr;
    const at::Tensor *w = router ? c.tensor(2, c.type, {router->size(0), -1, x->size(1)}) : nullptr;
    if (!w || w->size(1) % 2) return nothing();
    const int64_t M = x->size(0), D = x->size(1), E = router->size(0), F = w->size(1) / 2;
    const at::Tensor *down = c.tensor(3, c.type, {E, D, F});
    const int64_t top_k = c.integer(4);
    const bool normalize = c.truth(5);
    const int act = (int)c.integer(6);
    const bool routing = c.truth(7);
    if (!c.ok || top_k < 1 || top_k > E) return nothing();
    at::Tensor y = made(x, c.type, {M, D}), experts, weights;
    if (routing) {
      experts = made(x, at::kInt, {M, top_k});
      weights = made(x, at::kFloat, {M, top_k});
    }
    const auto f = reinterpret_cast<decltype(&pgemm_f16_moe)>(c.entry);
    if (f(ptr(x), ptr(router), ptr(w), ptr(down), ptr(&y), routing ? ptr<int32_t>(&experts) : nullptr,
          routing ? ptr<float>(&weights) : nullptr, M, E, D, F, top_k, normalize, act, c.stream) != PGEMM_OK)
      return nothing();
    if (!routing) return THPVariable_Wrap(std::move(y));
    PyObject *t = PyTuple_New(3);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(y)));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(experts)));
    PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(std::move(weights)));
    return t;
  });
}

// logits, u, temperature, top_k, top_p, min_p (each of these or None)
PyObject *sample(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c(args, n, 6);
    const at::Tensor *z = c.ok ? c.tensor(0, c.type, {-1, -1}) : nullptr;
    if (!c.ok) return nothing();
    const int64_t M = z->size(0), V = z->size(1);
    const at::Tensor *u = c.tensor(1, at::kFloat, {M});
    const void *settings[4];
    int shared = 0;
    for (int i = 0; i < 4; ++i) {
      settings[i] = nullptr;
      if (!c.ok || c.none(2 + i)) continue;
      if (!THPVariable_Check(args[kFixed + 2 + i])) return nothing();
      const bool one = THPVariable_Unpack(args[kFixed + 2 + i]).dim() == 0;
      const ScalarType st = i == 1 ? at::kInt : at::kFloat;
      const at::Tensor *t = one ? c.tensor(2 + i, st, {}) : c.tensor(2 + i, st, {M});
      if (!t) return nothing();
      settings[i] = t->data_ptr();
      shared |= one ? 1 << i : 0;
    }
    if (!c.ok) return nothing();
    at::Tensor token = made(z, at::kLong, {M});
    const auto f = reinterpret_cast<decltype(&pgemm_f16_sample)>(c.entry);
    if (f(ptr(z), ptr<float>(u), static_cast<const float *>(settings[0]), static_cast<const int32_t *>(settings[1]),
          static_cast<const float *>(settings[2]), static_cast<const float *>(settings[3]), shared, ptr<int64_t>(&token), M, V,
          c.stream) != PGEMM_OK)
      return nothing();
    return THPVariable_Wrap(std::move(token));
  });
}

#define METHOD(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(gated),  METHOD(gated_bwd), METHOD(xent),      METHOD(xent_bwd),
                         METHOD(q4),     METHOD(q4_gated),  METHOD(quant_i8),  METHOD(i8),
                         METHOD(i8_gated), METHOD(moe),     METHOD(sample),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
