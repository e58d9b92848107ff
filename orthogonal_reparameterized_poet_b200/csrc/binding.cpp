// The common call of the operators around the blocks (poet_joint_*,
// poet_token_logprobs*, poet_distill_topk*) on torch tensors, without the
// interpreter's part in it: looking through a call's tensors and allocating its
// results costs about 10 us in Python, several times the kernel of a small call.
//
// Every function takes its arguments by position and returns its result; None
// where an operand is anything but a contiguous tensor of the expected type and
// shape on the current device (the caller then looks at it in detail, and either
// passes its strides on or says what is wrong); or the library's status, an int,
// where the library refuses the call.  Calls run on the current stream.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <optional>

#include "poet.h"

namespace {

using at::Tensor;
using Args = PyObject *const *;

// A tensor argument; nullptr for None.  Sets ok to false for anything else.
const Tensor *tensor(PyObject *a, bool &ok) {
  if (a == Py_None) return nullptr;
  if (!THPVariable_Check(a)) {
    ok = false;
    return nullptr;
  }
  return &THPVariable_Unpack(a);
}

// Whether t is contiguous, of this type and on device dev.
bool plain(const Tensor &t, at::ScalarType type, int dev) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.layout() == at::kStrided && t.is_contiguous() &&
         !t.is_conj() && !t.is_neg();
}
bool plain1(const Tensor &t, at::ScalarType type, int dev, int64_t n) {
  return plain(t, type, dev) && t.dim() == 1 && t.size(0) == n;
}
bool plain2(const Tensor &t, at::ScalarType type, int dev, int64_t n, int64_t m) {
  return plain(t, type, dev) && t.dim() == 2 && t.size(0) == n && t.size(1) == m;
}
// The current device if t is a float32 or bfloat16 matrix on it, -1 otherwise.
int matrix(const Tensor *t) {
  if (!t || !t->is_cuda() || t->dim() != 2 || t->size(1) > INT32_MAX) return -1;
  const auto type = t->scalar_type();
  const int dev = int(c10::cuda::current_device());
  return (type == at::kBFloat16 || type == at::kFloat) && plain(*t, type, dev) ? dev : -1;
}
int32_t dtype_of(const Tensor &t) { return t.scalar_type() == at::kBFloat16 ? POET_BF16 : POET_F32; }
void *at_(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
template <typename T>
T *at_as(const Tensor *t) { return static_cast<T *>(at_(t)); }
poet_stream stream_of(int dev) { return reinterpret_cast<poet_stream>(c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream()); }

// On near's device, without torch's dispatch, which takes longer than the allocation.
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor &near) {
  return Tensor(at::detail::empty_cuda(shape, type, near.device(), std::nullopt));
}
PyObject *wrap(const std::optional<Tensor> &t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}
template <size_t N>
PyObject *wrap(const std::optional<Tensor> (&t)[N]) {
  PyObject *r = PyTuple_New(N);
  if (!r) return nullptr;
  for (size_t i = 0; i < N; ++i) {
    PyObject *o = wrap(t[i]);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}
// Runs f without the interpreter's lock: other Python threads run while this one
// allocates and launches, which may both wait for the GPU.  f touches no object of
// the interpreter's; the caller's frame holds the tensors that it reads.
template <typename F>
poet_status unlocked(F f) {
  struct Lock {
    PyThreadState *state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return f();
}

PyObject *status(poet_status s) { return PyLong_FromLong(long(s)); }
const Tensor *given(const std::optional<Tensor> &t) { return t ? &*t : nullptr; }

// No C++ exception leaves to the interpreter (an allocation may throw).
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    PyObject *r = f();
    if (PyErr_Occurred()) {
      Py_XDECREF(r);
      return nullptr;
    }
    return r;
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *torch = PyImport_ImportModule("torch"), *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown exception");
  }
  return nullptr;
}

// A joint's operands after h (the stream, or the forward's result): o, the gate
// and the gains; false if any is not plain.
struct Joint {
  poet_joint J{};
  int dev = -1;
  int64_t T = 0, d = 0, G = 0;
  const Tensor *o = nullptr, *h = nullptr, *gate = nullptr, *w_post = nullptr, *w_pre = nullptr;
  at::ScalarType type = at::kFloat;
  int64_t ldg = 0;
  // options: post_norm, gate_act, gate_rows, alpha, beta, eps
  bool take(PyObject *po, PyObject *ph, PyObject *pg, PyObject *pq, PyObject *pn, Args options) {
    bool ok = true;
    o = tensor(po, ok);
    h = tensor(ph, ok);
    gate = tensor(pg, ok);
    w_post = tensor(pq, ok);
    w_pre = tensor(pn, ok);
    dev = ok && o ? matrix(h) : -1;
    if (dev < 0) return false;
    T = h->size(0);
    d = h->size(1);
    type = h->scalar_type();
    J.d = int32_t(d);
    J.dtype = dtype_of(*h);
    const int post = PyObject_IsTrue(options[0]);
    const long long act = PyLong_AsLongLong(options[1]), rows = PyLong_AsLongLong(options[2]);
    J.post_norm = post == 1;
    J.gate_act = act < INT32_MIN || act > INT32_MAX ? -1 : int32_t(act);
    J.gate_rows = rows;
    J.alpha = float(PyFloat_AsDouble(options[3]));
    J.beta = float(PyFloat_AsDouble(options[4]));
    J.eps = float(PyFloat_AsDouble(options[5]));
    if (PyErr_Occurred() || rows < 1) return false;
    if (!plain2(*o, type, dev, T, d) || (w_post && !plain1(*w_post, at::kFloat, dev, d)) ||
        (w_pre && !plain1(*w_pre, at::kFloat, dev, d)))
      return false;
    if (gate) {
      G = T / rows + (T % rows ? 1 : 0);
      if (gate->dim() == 2 ? !plain2(*gate, type, dev, G, d) : !plain1(*gate, type, dev, G)) return false;
      J.gate = gate->dim() == 2 ? POET_GATE_CHANNEL : POET_GATE_ROW;
      ldg = gate->dim() == 2 ? d : 1;
    }
    J.w_post = at_as<float>(w_post);
    J.w_pre = at_as<float>(w_pre);
    return true;
  }
};

// (o, h, gate, w_post, w_pre, post_norm, gate_act, gate_rows, alpha, beta, eps, pre_norm)
PyObject *joint_forward(PyObject *, Args a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject * {
    Joint j;
    if (!j.take(a[0], a[1], a[2], a[3], a[4], a + 5)) Py_RETURN_NONE;
    const bool pre = PyObject_IsTrue(a[11]) == 1;
    std::optional<Tensor> out[2];
    const poet_status s = unlocked([&] {
      out[0] = fresh({j.T, j.d}, j.type, *j.h);
      if (pre) out[1] = fresh({j.T, j.d}, j.type, *j.h);
      return poet_joint_forward(&j.J, at_(j.o), j.d, at_(j.h), j.d, at_(j.gate), j.ldg, j.T, at_(given(out[0])), j.d,
                                at_(given(out[1])), j.d, stream_of(j.dev));
    });
    return s == POET_OK ? wrap(out) : status(s);
  });
}

// (o, h_out, gate, w_post, w_pre, post_norm, gate_act, gate_rows, alpha, beta, eps, dh_out, dn)
PyObject *joint_backward(PyObject *, Args a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    Joint j;
    if (!j.take(a[0], a[1], a[2], a[3], a[4], a + 5)) Py_RETURN_NONE;
    bool ok = true;
    const Tensor *dh_out = tensor(a[11], ok), *dn = tensor(a[12], ok);
    if (!ok || (dh_out && !plain2(*dh_out, j.type, j.dev, j.T, j.d)) || (dn && !plain2(*dn, j.type, j.dev, j.T, j.d)) ||
        (!dn && j.w_pre))
      Py_RETURN_NONE;
    std::optional<Tensor> out[5];  // dh, d_o, dgate, dw_post, dw_pre
    const poet_status s = unlocked([&] {
      out[0] = fresh({j.T, j.d}, j.type, *j.h);
      out[1] = fresh({j.T, j.d}, j.type, *j.h);
      if (j.gate) out[2] = fresh(j.gate->sizes(), j.type, *j.h);
      if (j.w_post) out[3] = fresh({j.d}, at::kFloat, *j.h);
      if (j.w_pre) out[4] = fresh({j.d}, at::kFloat, *j.h);
      const size_t bytes = poet_joint_workspace_bytes(&j.J, j.T);
      const Tensor ws = fresh({int64_t(bytes ? bytes : 1)}, at::kByte, *j.h);
      return poet_joint_backward(&j.J, at_(j.o), j.d, at_(j.h), j.d, at_(j.gate), j.ldg, at_(dh_out), j.d, at_(dn), j.d, j.T,
                                 at_(given(out[0])), j.d, at_(given(out[1])), j.d, at_(given(out[2])), j.ldg,
                                 at_as<float>(given(out[3])), at_as<float>(given(out[4])), at_(&ws), bytes,
                                 stream_of(j.dev));
    });
    return s == POET_OK ? wrap(out) : status(s);
  });
}

// One value of this type per row, or None.
bool per_row(const Tensor *t, at::ScalarType type, int dev, int64_t T) { return !t || plain1(*t, type, dev, T); }

// (logits, tokens, topk, scale, entropy)
PyObject *token_logprobs(PyObject *, Args a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    bool ok = true;
    const Tensor *x = tensor(a[0], ok), *tokens = tensor(a[1], ok);
    const int dev = ok ? matrix(x) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const int64_t T = x->size(0), V = x->size(1);
    const long long topk = PyLong_AsLongLong(a[2]);
    const float scale = float(PyFloat_AsDouble(a[3]));
    if (PyErr_Occurred()) return nullptr;
    if (!per_row(tokens, at::kInt, dev, T) || topk < 0 || topk > INT32_MAX) Py_RETURN_NONE;
    const bool entropy = PyObject_IsTrue(a[4]) == 1;
    std::optional<Tensor> out[5];  // logp, entropy, top_tokens, top_logp, saved
    const poet_status s = unlocked([&] {
      if (tokens) out[0] = fresh({T}, at::kFloat, *x);
      if (entropy) out[1] = fresh({T}, at::kFloat, *x);
      if (topk > 0) {
        out[2] = fresh({T, topk}, at::kInt, *x);
        out[3] = fresh({T, topk}, at::kFloat, *x);
      }
      out[4] = fresh({T, 4}, at::kFloat, *x);
      return poet_token_logprobs(at_(x), V, dtype_of(*x), T, int32_t(V), scale, at_as<int32_t>(tokens), int32_t(topk),
                                 at_as<float>(given(out[0])), at_as<float>(given(out[1])), at_as<int32_t>(given(out[2])),
                                 at_as<float>(given(out[3])), at_as<float>(given(out[4])), stream_of(dev));
    });
    return s == POET_OK ? wrap(out) : status(s);
  });
}

// (logits, tokens, saved, dlogp, dentropy, scale)
PyObject *token_logprobs_grad(PyObject *, Args a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject * {
    bool ok = true;
    const Tensor *x = tensor(a[0], ok), *tokens = tensor(a[1], ok), *saved = tensor(a[2], ok), *dlogp = tensor(a[3], ok),
                 *dentropy = tensor(a[4], ok);
    const int dev = ok && saved ? matrix(x) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const int64_t T = x->size(0), V = x->size(1);
    const float scale = float(PyFloat_AsDouble(a[5]));
    if (PyErr_Occurred()) return nullptr;
    if (!per_row(tokens, at::kInt, dev, T) || !plain2(*saved, at::kFloat, dev, T, 4) || !per_row(dlogp, at::kFloat, dev, T) ||
        !per_row(dentropy, at::kFloat, dev, T))
      Py_RETURN_NONE;
    std::optional<Tensor> out;
    const poet_status s = unlocked([&] {
      out = fresh({T, V}, x->scalar_type(), *x);
      return poet_token_logprobs_grad(at_(x), V, dtype_of(*x), T, int32_t(V), scale, at_as<int32_t>(tokens),
                                      at_as<float>(saved), at_as<float>(dlogp), at_as<float>(dentropy), at_(given(out)), V,
                                      stream_of(dev));
    });
    return s == POET_OK ? wrap(out) : status(s);
  });
}

// The teacher's entries of T rows; their number, or -1.
int64_t teacher(const Tensor *tokens, const Tensor *values, int dev, int64_t T) {
  if (!tokens || !values || tokens->dim() != 2 || tokens->size(1) > INT32_MAX) return -1;
  const int64_t K = tokens->size(1);
  return plain2(*tokens, at::kInt, dev, T, K) && plain2(*values, at::kFloat, dev, T, K) ? K : -1;
}

// (logits, teacher_tokens, teacher_values, value_scale, tail, scale, dloss, grad)
PyObject *distill_topk(PyObject *, Args a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    bool ok = true;
    const Tensor *x = tensor(a[0], ok), *tokens = tensor(a[1], ok), *values = tensor(a[2], ok), *dloss = tensor(a[6], ok);
    const int dev = ok ? matrix(x) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const int64_t T = x->size(0), V = x->size(1), K = teacher(tokens, values, dev, T);
    const float value_scale = float(PyFloat_AsDouble(a[3])), scale = float(PyFloat_AsDouble(a[5]));
    const int tail = PyObject_IsTrue(a[4]), grad = PyObject_IsTrue(a[7]);
    if (PyErr_Occurred()) return nullptr;
    if (K < 0 || !per_row(dloss, at::kFloat, dev, T)) Py_RETURN_NONE;
    std::optional<Tensor> out[3];  // loss, dlogits, saved
    const poet_status s = unlocked([&] {
      out[0] = fresh({T}, at::kFloat, *x);
      if (grad == 1) out[1] = fresh({T, V}, x->scalar_type(), *x);
      out[2] = fresh({T, 4}, at::kFloat, *x);
      return poet_distill_topk(at_(x), V, dtype_of(*x), T, int32_t(V), scale, at_as<int32_t>(tokens), at_as<float>(values),
                               int32_t(K), value_scale, tail == 1, at_as<float>(dloss), at_as<float>(given(out[0])),
                               at_as<float>(given(out[2])), at_(given(out[1])), V, stream_of(dev));
    });
    return s == POET_OK ? wrap(out) : status(s);
  });
}

// (logits, teacher_tokens, teacher_values, value_scale, tail, scale, saved, dloss)
PyObject *distill_topk_grad(PyObject *, Args a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    bool ok = true;
    const Tensor *x = tensor(a[0], ok), *tokens = tensor(a[1], ok), *values = tensor(a[2], ok), *saved = tensor(a[6], ok),
                 *dloss = tensor(a[7], ok);
    const int dev = ok && saved ? matrix(x) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const int64_t T = x->size(0), V = x->size(1), K = teacher(tokens, values, dev, T);
    const float value_scale = float(PyFloat_AsDouble(a[3])), scale = float(PyFloat_AsDouble(a[5]));
    const int tail = PyObject_IsTrue(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (K < 0 || !plain2(*saved, at::kFloat, dev, T, 4) || !per_row(dloss, at::kFloat, dev, T)) Py_RETURN_NONE;
    std::optional<Tensor> out;
    const poet_status s = unlocked([&] {
      out = fresh({T, V}, x->scalar_type(), *x);
      return poet_distill_topk_grad(at_(x), V, dtype_of(*x), T, int32_t(V), scale, at_as<int32_t>(tokens),
                                    at_as<float>(values), int32_t(K), value_scale, tail == 1, at_as<float>(saved),
                                    at_as<float>(dloss), at_(given(out)), V, stream_of(dev));
    });
    return s == POET_OK ? wrap(out) : status(s);
  });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(joint_forward),       METHOD(joint_backward), METHOD(token_logprobs),
                         METHOD(token_logprobs_grad), METHOD(distill_topk),   METHOD(distill_topk_grad),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
