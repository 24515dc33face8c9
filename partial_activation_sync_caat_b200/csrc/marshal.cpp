// marshal.cpp - the Python binding's marshalling of the attention block's calls, compiled: a call on
// small tensors takes less time on the GPU than the interpreter needs to look up their addresses,
// shapes and strides (rotary positions of 8 tokens with an
// append: 11.0 us a call through the interpreter's accessors, 4.3 with this).
//
// Every function returns the library's status, or None for arguments it does not take (another type,
// shape, device or layout than the ordinary one): the binding then goes through its own checks, which
// name what is wrong.  Nothing is kept between calls.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <vector>

#include "caat.h"

namespace {

struct Library {
  decltype(&caat_rope) rope;
  decltype(&caat_attn_forward) forward;
  decltype(&caat_attn_backward) backward;
  decltype(&caat_attn_decode) decode;
  decltype(&caat_attn_workspace_size) workspace_size;
} lib;

const at::Tensor* tensor(PyObject* o, int dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == dev ? &t : nullptr;
}

// Device of the first tensor, -1 if that is not the current one.
int device_of(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return -1;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.get_device() == c10::cuda::current_device() ? t.get_device() : -1;
}

// A contiguous tensor of that type and shape.
template <class T>
bool like(PyObject* o, at::ScalarType type, c10::IntArrayRef shape, int dev, T** p) {
  const at::Tensor* t = tensor(o, dev);
  if (!t || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous()) return false;
  *p = static_cast<T*>(t->data_ptr());
  return true;
}

// bf16 [P, T, heads, dh] whose heads lie side by side within a token: address and (rank, token) strides,
// 0 for a contiguous tensor, and for no other.
bool heads4(const at::Tensor* t, const caat_bf16** p, int64_t* rank, int64_t* token) {
  if (!t || t->dim() != 4 || t->scalar_type() != at::kBFloat16) return false;
  *p = static_cast<const caat_bf16*>(t->data_ptr());
  *rank = *token = 0;
  if (t->is_contiguous()) return true;
  const auto n = t->sizes(), s = t->strides();
  if ((n[3] > 1 && s[3] != 1) || (n[2] > 1 && s[2] != n[3])) return false;
  *token = n[1] > 1 ? s[1] : n[2] * n[3];  // a dimension of one element has no stride of its own
  if (*token < n[2] * n[3]) return false;  // an expanded tensor: (0, 0) would mean contiguous
  *rank = n[0] > 1 ? s[0] : std::max(s[0], *token * n[1]);
  return true;
}

// A rotation's output: contiguous, or the input itself.
bool rope_out(PyObject* o, const at::Tensor& x, int dev, caat_bf16** p) {
  const at::Tensor* t = tensor(o, dev);
  if (!t) return false;
  if (t->data_ptr() == x.data_ptr() && x.numel() > 0) {
    *p = static_cast<caat_bf16*>(t->data_ptr());
    return t->scalar_type() == at::kBFloat16 && t->sizes() == x.sizes() && t->strides() == x.strides();
  }
  return like(o, at::kBFloat16, x.sizes(), dev, p);
}

// Host int32 offsets: the values of a list or tuple, or a one-dimensional int32 array in place.
struct Offsets {
  std::vector<int32_t> values;
  Py_buffer view{};
  const int32_t* p = nullptr;
  int64_t n = 0;
  ~Offsets() {
    if (view.obj) PyBuffer_Release(&view);
  }
  bool read(PyObject* o) {
    if (PyList_CheckExact(o) || PyTuple_CheckExact(o)) {
      n = PySequence_Fast_GET_SIZE(o);
      values.resize(n);
      for (int64_t i = 0; i < n; ++i) {
        PyObject* x = PySequence_Fast_GET_ITEM(o, i);
        int over = 0;
        if (!PyLong_CheckExact(x)) return false;
        const long v = PyLong_AsLongAndOverflow(x, &over);
        if (over || v < INT32_MIN || v > INT32_MAX) return false;
        values[i] = static_cast<int32_t>(v);
      }
      p = values.data();
    } else {
      if (!PyObject_CheckBuffer(o)) return false;
      if (PyObject_GetBuffer(o, &view, PyBUF_ND | PyBUF_FORMAT | PyBUF_C_CONTIGUOUS) != 0) {
        PyErr_Clear();
        return false;
      }
      if (view.ndim != 1 || !view.format || std::strcmp(view.format, "i") != 0) return false;
      n = view.shape[0];
      p = static_cast<const int32_t*>(view.buf);
    }
    return n > 0;
  }
};

bool number(PyObject* o, double* v) {
  if (!PyFloat_CheckExact(o)) return false;
  *v = PyFloat_AS_DOUBLE(o);
  return true;
}

bool scale_of(PyObject* o, int64_t dh, float* scale) {
  double v = dh > 0 ? std::pow(static_cast<double>(dh), -0.5) : 0.0;
  if (o != Py_None && !number(o, &v)) return false;
  *scale = static_cast<float>(v);
  return true;
}

bool ints(std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x < 0 || x > INT32_MAX) return false;
  return true;
}

// The caller's workspace, if it gave one.
template <class Args>
bool given_workspace(PyObject* o, int dev, Args* a) {
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, dev);
  if (!t || !t->is_contiguous()) return false;  // (its elements say how long it is)
  a->workspace = t->data_ptr();
  a->ws_bytes = static_cast<size_t>(t->numel()) * t->element_size();
  return true;
}

template <class Args>
caat_status unlocked(caat_status (*call)(const Args*), const Args* a) {
  caat_status s;
  Py_BEGIN_ALLOW_THREADS s = call(a);
  Py_END_ALLOW_THREADS return s;
}

// The call; where it asks for a workspace and the caller gave none, once more with one of its own.
template <class Args>
PyObject* finish(caat_status (*call)(const Args*), Args* a, PyObject* workspace, int dev, int64_t Tq, int64_t Tk, int n_seq, int variant) {
  a->stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  caat_status s = unlocked(call, a);
  if (s == CAAT_ERR_WORKSPACE && workspace == Py_None) {
    const size_t need = lib.workspace_size(Tq, Tk, n_seq, a->P, a->heads_q, a->heads_k, a->dh, variant);
    const at::Tensor ws = at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev));
    a->workspace = ws.data_ptr();
    a->ws_bytes = need;
    s = unlocked(call, a);
  }
  return PyLong_FromLong(s);
}

// rope(q, k, v, positions, slots, inv_freq, q_out, k_out, v_out, interleaved, backward, mscale)
PyObject* rope(PyObject*, PyObject* const* x, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12 || !lib.rope) Py_RETURN_NONE;
  PyObject *q = x[0], *k = x[1], *positions = x[3], *slots = x[4];
  const int dev = device_of(q != Py_None ? q : k);
  if (dev < 0) Py_RETURN_NONE;
  caat_rope_args a{};
  const at::Tensor *tq = nullptr, *tk = nullptr;
  if (q != Py_None) {
    tq = tensor(q, dev);
    if (!heads4(tq, &a.q, &a.q_stride_rank, &a.q_stride_token) || !rope_out(x[6], *tq, dev, &a.q_out)) Py_RETURN_NONE;
    a.heads_q = static_cast<int32_t>(tq->size(2));
  }
  if (k != Py_None) {
    tk = tensor(k, dev);
    if (!heads4(tk, &a.k, &a.k_stride_rank, &a.k_stride_token)) Py_RETURN_NONE;
    if (tq && (tk->size(0) != tq->size(0) || tk->size(1) != tq->size(1) || tk->size(3) != tq->size(3))) Py_RETURN_NONE;
    a.heads_k = static_cast<int32_t>(tk->size(2));
  }
  const at::Tensor& first = tq ? *tq : *tk;
  const int64_t P = first.size(0), T = first.size(1), dh = first.size(3);
  if (!ints({P, dh, first.size(2), a.heads_q, a.heads_k})) Py_RETURN_NONE;
  if (tk && slots == Py_None && !rope_out(x[7], *tk, dev, &a.k_out)) Py_RETURN_NONE;
  if (slots != Py_None) {
    if (!tk) Py_RETURN_NONE;
    const at::Tensor *tv = tensor(x[2], dev), *cache = tensor(x[7], dev);
    if (!heads4(tv, &a.v, &a.v_stride_rank, &a.v_stride_token) || tv->sizes() != tk->sizes() || !cache) Py_RETURN_NONE;
    const auto c = cache->sizes();
    const size_t d = c.size();
    if ((d != 4 && d != 5) || c[0] != P || c[d - 2] != a.heads_k || c[d - 1] != dh) Py_RETURN_NONE;
    a.cache_rows = d == 5 ? c[1] * c[2] : c[1];
    if (!like(x[7], at::kBFloat16, c, dev, &a.k_out) || !like(x[8], at::kBFloat16, c, dev, &a.v_out) ||
        !like(slots, at::kLong, {T}, dev, &a.slots))
      Py_RETURN_NONE;
  }
  if (positions != Py_None && !like(positions, at::kInt, {T}, dev, &a.positions)) Py_RETURN_NONE;
  double mscale = 1.0;
  if (!number(x[11], &mscale) || !PyBool_Check(x[9]) || !PyBool_Check(x[10])) Py_RETURN_NONE;
  Py_buffer freq{};
  if (!PyObject_CheckBuffer(x[5])) Py_RETURN_NONE;
  if (PyObject_GetBuffer(x[5], &freq, PyBUF_ND | PyBUF_FORMAT | PyBUF_C_CONTIGUOUS) != 0) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  struct Release {
    Py_buffer* b;
    ~Release() { PyBuffer_Release(b); }
  } release{&freq};
  if (freq.ndim != 1 || !freq.format || std::strcmp(freq.format, "d") != 0 || freq.shape[0] > INT32_MAX / 2) Py_RETURN_NONE;
  a.inv_freq = static_cast<const double*>(freq.buf);
  a.rot = static_cast<int32_t>(2 * freq.shape[0]);
  a.P = static_cast<int32_t>(P);
  a.T = T;
  a.dh = static_cast<int32_t>(dh);
  a.mscale = static_cast<float>(mscale);
  a.flags = (x[9] == Py_True ? CAAT_ROPE_FLAG_INTERLEAVED : 0u) | (x[10] == Py_True ? CAAT_ROPE_FLAG_BACKWARD : 0u);
  a.stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  return PyLong_FromLong(unlocked(lib.rope, &a));
  END_HANDLE_TH_ERRORS
}

// What the forward and the backward share: q, k, v, cu_q, cu_k.
template <class Args>
bool qkv(PyObject* const* x, int dev, Args* a, Offsets* cq, Offsets* ck, const at::Tensor** tq, const at::Tensor** tk) {
  *tq = tensor(x[0], dev);
  *tk = tensor(x[1], dev);
  const at::Tensor* tv = tensor(x[2], dev);
  if (!heads4(*tq, &a->q, &a->q_stride_rank, &a->q_stride_token) || !heads4(*tk, &a->k, &a->k_stride_rank, &a->k_stride_token) ||
      !heads4(tv, &a->v, &a->v_stride_rank, &a->v_stride_token) || tv->sizes() != (*tk)->sizes())
    return false;
  const auto q = (*tq)->sizes(), k = (*tk)->sizes();
  if (k[0] != q[0] || k[3] != q[3] || !ints({q[0], q[2], q[3], k[2]}) || !cq->read(x[3])) return false;
  if (x[4] != Py_None && (!ck->read(x[4]) || ck->n != cq->n)) return false;
  if (cq->n - 1 > INT32_MAX) return false;
  a->cu_q = cq->p;
  a->cu_k = ck->p;
  a->n_seq = static_cast<int32_t>(cq->n - 1);
  a->P = static_cast<int32_t>(q[0]);
  a->Tq = q[1];
  a->Tk = k[1];
  a->heads_q = static_cast<int32_t>(q[2]);
  a->heads_k = static_cast<int32_t>(k[2]);
  a->dh = static_cast<int32_t>(q[3]);
  return true;
}

// attn_forward(q, k, v, cu_q, cu_k, out, lse, scale, workspace)
PyObject* attn_forward(PyObject*, PyObject* const* x, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9 || !lib.forward) Py_RETURN_NONE;
  const int dev = device_of(x[0]);
  caat_attn_args a{};
  Offsets cq, ck;
  const at::Tensor *tq, *tk;
  if (dev < 0 || !qkv(x, dev, &a, &cq, &ck, &tq, &tk)) Py_RETURN_NONE;
  if (!like(x[5], at::kBFloat16, {a.P, a.Tq, int64_t(a.heads_q) * a.dh}, dev, &a.out) ||
      (x[6] != Py_None && !like(x[6], at::kFloat, {a.P, a.heads_q, a.Tq}, dev, &a.lse)) || !scale_of(x[7], a.dh, &a.scale) ||
      !given_workspace(x[8], dev, &a))
    Py_RETURN_NONE;
  return finish(lib.forward, &a, x[8], dev, a.Tq, a.Tk, a.n_seq, CAAT_VARIANT_ATTN);
  END_HANDLE_TH_ERRORS
}

// attn_backward(q, k, v, cu_q, cu_k, out, lse, dout, dq, dk, dv, scale, workspace)
PyObject* attn_backward(PyObject*, PyObject* const* x, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 13 || !lib.backward) Py_RETURN_NONE;
  const int dev = device_of(x[0]);
  caat_attn_bwd_args a{};
  Offsets cq, ck;
  const at::Tensor *tq, *tk;
  if (dev < 0 || !qkv(x, dev, &a, &cq, &ck, &tq, &tk)) Py_RETURN_NONE;
  const int64_t rows[3] = {a.P, a.Tq, int64_t(a.heads_q) * a.dh};
  if (!like(x[5], at::kBFloat16, rows, dev, &a.out) || !like(x[6], at::kFloat, {a.P, a.heads_q, a.Tq}, dev, &a.lse) ||
      !like(x[7], at::kBFloat16, rows, dev, &a.dout) || !like(x[8], at::kBFloat16, tq->sizes(), dev, &a.dq) ||
      !like(x[9], at::kBFloat16, tk->sizes(), dev, &a.dk) || !like(x[10], at::kBFloat16, tk->sizes(), dev, &a.dv) ||
      !scale_of(x[11], a.dh, &a.scale) || !given_workspace(x[12], dev, &a))
    Py_RETURN_NONE;
  return finish(lib.backward, &a, x[12], dev, a.Tq, a.Tk, a.n_seq, CAAT_VARIANT_ATTN_BWD);
  END_HANDLE_TH_ERRORS
}

// attn_decode(q, k_cache, v_cache, lens, out, scale, workspace)
PyObject* attn_decode(PyObject*, PyObject* const* x, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7 || !lib.decode) Py_RETURN_NONE;
  const int dev = device_of(x[0]);
  if (dev < 0) Py_RETURN_NONE;
  caat_attn_decode_args a{};
  const at::Tensor *tq = tensor(x[0], dev), *cache = tensor(x[1], dev);
  if (!heads4(tq, &a.q, &a.q_stride_rank, &a.q_stride_token) || !cache || cache->dim() != 5) Py_RETURN_NONE;
  const auto q = tq->sizes(), c = cache->sizes();
  if (c[0] != q[0] || c[1] != q[1] || c[4] != q[3] || !ints({q[0], q[2], q[3], c[3]})) Py_RETURN_NONE;
  a.P = static_cast<int32_t>(q[0]);
  a.B = q[1];
  a.capacity = c[2];
  a.heads_q = static_cast<int32_t>(q[2]);
  a.heads_k = static_cast<int32_t>(c[3]);
  a.dh = static_cast<int32_t>(q[3]);
  if (!like(x[1], at::kBFloat16, c, dev, &a.k_cache) || !like(x[2], at::kBFloat16, c, dev, &a.v_cache) ||
      !like(x[3], at::kInt, {a.B}, dev, &a.lens) || !like(x[4], at::kBFloat16, {a.P, a.B, int64_t(a.heads_q) * a.dh}, dev, &a.out) ||
      !scale_of(x[5], a.dh, &a.scale) || !given_workspace(x[6], dev, &a))
    Py_RETURN_NONE;
  return finish(lib.decode, &a, x[6], dev, a.B, a.capacity, 0, CAAT_VARIANT_ATTN_DECODE);
  END_HANDLE_TH_ERRORS
}

// bind(rope, attn_forward, attn_backward, attn_decode, attn_workspace_size): the library's functions
PyObject* bind(PyObject*, PyObject* const* x, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(x[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  lib.rope = reinterpret_cast<decltype(lib.rope)>(p[0]);
  lib.forward = reinterpret_cast<decltype(lib.forward)>(p[1]);
  lib.backward = reinterpret_cast<decltype(lib.backward)>(p[2]);
  lib.decode = reinterpret_cast<decltype(lib.decode)>(p[3]);
  lib.workspace_size = reinterpret_cast<decltype(lib.workspace_size)>(p[4]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(rope), FAST(attn_forward), FAST(attn_backward), FAST(attn_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
