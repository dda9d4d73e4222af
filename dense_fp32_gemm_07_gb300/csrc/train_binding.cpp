// train_binding.cpp -- the tensor calls of train.py for plain arguments, in native
// code: contiguous operands of one type on the current device, results that the
// call allocates, the current stream.  Such a call costs the host a few
// microseconds where the same checks and conversions in Python cost 10 to 40,
// which is most of a small call's time.
//
// Each function answers a result as train.py documents it, or the library's error
// code as an int, or None when an argument is not of that plain kind (strided,
// another stream, `out` given, wrong in some way); train.py then goes through its
// own checks, which serve it or say what is wrong.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#include "../../include/b2g_train.h"

namespace {

using at::Tensor;

// A call's element type and device, from its first operand.
struct Kind {
  at::ScalarType type;
  at::Device device{at::kCPU};
  int code;
  void* stream;

  bool take(const Tensor& t) {
    type = t.scalar_type();
    if (type == at::kFloat)
      code = B2G_F32;
    else if (type == at::kBFloat16)
      code = B2G_BF16;
    else
      return false;
    device = t.device();
    if (!device.is_cuda() || device.index() != c10::cuda::current_device()) return false;
    stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    return true;
  }
  bool has(const Tensor& t, at::ScalarType want) const {
    return t.scalar_type() == want && t.device() == device && t.is_contiguous();
  }
  bool matrix(const Tensor& t) const { return has(t, type) && t.dim() == 2; }
  bool vector(const Tensor& t, at::ScalarType want, int64_t n) const {
    return has(t, want) && t.dim() == 1 && t.size(0) == n;
  }
  // Row numbers: their width in bytes, 0 when they are not.
  int indices(const Tensor& t) const {
    if (t.dim() != 1 || t.device() != device || !t.is_contiguous()) return 0;
    return t.scalar_type() == at::kLong ? 8 : t.scalar_type() == at::kInt ? 4 : 0;
  }
  Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::empty(shape, at::TensorOptions().dtype(t).device(device));
  }
  Tensor empty(at::IntArrayRef shape) const { return empty(shape, type); }
  Tensor bytes(size_t n) const { return empty({(int64_t)n}, at::kByte); }
};

bool small(int64_t n) { return n <= 0x7fffffff; }
long long ld(int64_t cols) { return cols > 1 ? cols : 1; }
void* ptr(const Tensor& t) { return t.data_ptr(); }

bool is_tensor(PyObject* o) { return THPVariable_Check(o); }
bool is_tensor_or_none(PyObject* o) { return o == Py_None || THPVariable_Check(o); }

// The tensor of an argument; an undefined one for None.
const Tensor& tensor(PyObject* o) {
  static const Tensor none;
  return o == Py_None ? none : THPVariable_Unpack(o);
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

template <typename... T>
PyObject* answer(int rc, const T&... t) {
  if (rc) return PyLong_FromLong(rc);
  if constexpr (sizeof...(T) == 1) {
    return wrap(t...);
  } else {
    PyObject* tuple = PyTuple_New(sizeof...(T));
    if (!tuple) return nullptr;
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(tuple, i++, wrap(t)), ...);
    return tuple;
  }
}

bool number(PyObject* o, double* v) {
  if (PyFloat_CheckExact(o)) {
    *v = PyFloat_AS_DOUBLE(o);
    return true;
  }
  if (!PyLong_CheckExact(o)) return false;
  *v = PyLong_AsDouble(o);
  if (*v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

bool whole(PyObject* o, long long* v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}

// layer_norm(x, weight, bias, eps)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  double eps;
  if (n != 4 || !is_tensor(a[0]) || !is_tensor_or_none(a[1]) || !is_tensor_or_none(a[2]) ||
      !number(a[3], &eps))
    Py_RETURN_NONE;
  const Tensor &x = tensor(a[0]), &w = tensor(a[1]), &b = tensor(a[2]);
  Kind k;
  if (!k.take(x) || !k.matrix(x)) Py_RETURN_NONE;
  const int64_t r = x.size(0), c = x.size(1);
  if (!small(c) || c == 0 || (w.defined() && !k.vector(w, k.type, c)) ||
      (b.defined() && !k.vector(b, k.type, c)))
    Py_RETURN_NONE;
  const Tensor y = k.empty({r, c}), mean = k.empty({r}, at::kFloat), rstd = k.empty({r}, at::kFloat);
  const int rc = b2g_layernorm(k.code, r, (int)c, ptr(x), ld(c), w.defined() ? ptr(w) : nullptr,
                               b.defined() ? ptr(b) : nullptr, (float)eps, ptr(y), ld(c),
                               mean.data_ptr<float>(), rstd.data_ptr<float>(), k.stream);
  return answer(rc, y, mean, rstd);
  END_HANDLE_TH_ERRORS
}

// layer_norm_backward(dy, x, weight, mean, rstd, bias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6 || !is_tensor(a[0]) || !is_tensor(a[1]) || !is_tensor_or_none(a[2]) ||
      !is_tensor(a[3]) || !is_tensor(a[4]) || !PyBool_Check(a[5]))
    Py_RETURN_NONE;
  const Tensor &dy = tensor(a[0]), &x = tensor(a[1]), &w = tensor(a[2]), &mean = tensor(a[3]),
               &rstd = tensor(a[4]);
  Kind k;
  if (!k.take(x) || !k.matrix(x) || !k.matrix(dy) || dy.sizes() != x.sizes()) Py_RETURN_NONE;
  const int64_t r = x.size(0), c = x.size(1);
  if (!small(c) || (w.defined() && !k.vector(w, k.type, c)) || !k.vector(mean, at::kFloat, r) ||
      !k.vector(rstd, at::kFloat, r))
    Py_RETURN_NONE;
  size_t bytes = 0;
  int rc = b2g_layernorm_backward_workspace_size(k.code, r, (int)c, &bytes);
  if (rc) return answer(rc, x);
  const Tensor dx = k.empty({r, c}), dw = w.defined() ? k.empty({c}) : Tensor(),
               db = a[5] == Py_True ? k.empty({c}) : Tensor(), ws = k.bytes(bytes);
  rc = b2g_layernorm_backward(k.code, r, (int)c, ptr(dy), ld(c), ptr(x), ld(c),
                              w.defined() ? ptr(w) : nullptr, mean.data_ptr<float>(),
                              rstd.data_ptr<float>(), ptr(dx), ld(c),
                              dw.defined() ? ptr(dw) : nullptr, db.defined() ? ptr(db) : nullptr,
                              ptr(ws), bytes, k.stream);
  return answer(rc, dx, dw, db);
  END_HANDLE_TH_ERRORS
}

// embedding(ids, table, scale)
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  double scale;
  if (n != 3 || !is_tensor(a[0]) || !is_tensor(a[1]) || !number(a[2], &scale)) Py_RETURN_NONE;
  const Tensor &ids = tensor(a[0]), &table = tensor(a[1]);
  Kind k;
  if (!k.take(table) || !k.matrix(table)) Py_RETURN_NONE;
  const int width = k.indices(ids);
  const int64_t v = table.size(0), d = table.size(1);
  if (!width || !small(v) || !small(d)) Py_RETURN_NONE;
  const Tensor out = k.empty({ids.size(0), d});
  const int rc = b2g_embedding(k.code, ids.size(0), (int)v, (int)d, ptr(ids), width, ptr(table),
                               ld(d), (float)scale, ptr(out), ld(d), k.stream);
  return answer(rc, out);
  END_HANDLE_TH_ERRORS
}

// embedding_backward(ids, dout, num_rows, scale)
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  double scale;
  long long v;
  if (n != 4 || !is_tensor(a[0]) || !is_tensor(a[1]) || !whole(a[2], &v) || !number(a[3], &scale))
    Py_RETURN_NONE;
  const Tensor &ids = tensor(a[0]), &dout = tensor(a[1]);
  Kind k;
  if (!k.take(dout) || !k.matrix(dout)) Py_RETURN_NONE;
  const int width = k.indices(ids);
  const int64_t tokens = dout.size(0), d = dout.size(1);
  if (!width || ids.size(0) != tokens || v < 0 || !small(v) || !small(d)) Py_RETURN_NONE;
  size_t bytes = 0;
  int rc = b2g_embedding_backward_workspace_size(k.code, tokens, (int)v, (int)d, &bytes);
  if (rc) return answer(rc, dout);
  const Tensor out = k.empty({(int64_t)v, d}), ws = k.bytes(bytes);
  rc = b2g_embedding_backward(k.code, tokens, (int)v, (int)d, ptr(ids), width, ptr(dout), ld(d),
                              (float)scale, -1, 0, ptr(out), ld(d), ptr(ws), bytes, k.stream);
  return answer(rc, out);
  END_HANDLE_TH_ERRORS
}

// linear_cross_entropy(h, w, target, ignore_index)
PyObject* linear_cross_entropy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long long ignore;
  if (n != 4 || !is_tensor(a[0]) || !is_tensor(a[1]) || !is_tensor(a[2]) || !whole(a[3], &ignore))
    Py_RETURN_NONE;
  const Tensor &h = tensor(a[0]), &w = tensor(a[1]), &target = tensor(a[2]);
  Kind k;
  if (!k.take(h) || !k.matrix(h) || !k.matrix(w)) Py_RETURN_NONE;
  const int width = k.indices(target);
  const int64_t t = h.size(0), d = h.size(1), v = w.size(0);
  if (!width || w.size(1) != d || target.size(0) != t || !small(t) || !small(d) || !small(v))
    Py_RETURN_NONE;
  size_t bytes = 0;
  int rc = b2g_linear_xent_workspace_size(k.code, (int)t, (int)v, (int)d, ptr(h), ld(d), ptr(w),
                                          ld(d), 0, &bytes);
  if (rc) return answer(rc, h);
  const Tensor loss = k.empty({t}, at::kFloat), lse = k.empty({t}, at::kFloat), ws = k.bytes(bytes);
  rc = b2g_linear_xent(k.code, (int)t, (int)v, (int)d, ptr(h), ld(d), ptr(w), ld(d), ptr(target),
                       width, ignore, loss.data_ptr<float>(), lse.data_ptr<float>(), ptr(ws), bytes,
                       k.stream);
  return answer(rc, loss, lse);
  END_HANDLE_TH_ERRORS
}

// linear_cross_entropy_backward(h, w, target, lse, grad_loss, ignore_index)
PyObject* linear_cross_entropy_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long long ignore;
  if (n != 6 || !is_tensor(a[0]) || !is_tensor(a[1]) || !is_tensor(a[2]) || !is_tensor(a[3]) ||
      !is_tensor(a[4]) || !whole(a[5], &ignore))
    Py_RETURN_NONE;
  const Tensor &h = tensor(a[0]), &w = tensor(a[1]), &target = tensor(a[2]), &lse = tensor(a[3]),
               &g = tensor(a[4]);
  Kind k;
  if (!k.take(h) || !k.matrix(h) || !k.matrix(w)) Py_RETURN_NONE;
  const int width = k.indices(target);
  const int64_t t = h.size(0), d = h.size(1), v = w.size(0);
  if (!width || w.size(1) != d || target.size(0) != t || !k.vector(lse, at::kFloat, t) ||
      !k.vector(g, at::kFloat, t) || !small(t) || !small(d) || !small(v))
    Py_RETURN_NONE;
  size_t bytes = 0;
  int rc = b2g_linear_xent_workspace_size(k.code, (int)t, (int)v, (int)d, ptr(h), ld(d), ptr(w),
                                          ld(d), 1, &bytes);
  if (rc) return answer(rc, h);
  const Tensor dh = k.empty({t, d}), dw = k.empty({v, d}), ws = k.bytes(bytes);
  rc = b2g_linear_xent_backward(k.code, (int)t, (int)v, (int)d, ptr(h), ld(d), ptr(w), ld(d),
                                ptr(target), width, ignore, lse.data_ptr<float>(),
                                g.data_ptr<float>(), ptr(dh), ld(d), 0, ptr(dw), ld(d), ptr(ws),
                                bytes, k.stream);
  return answer(rc, dh, dw);
  END_HANDLE_TH_ERRORS
}

// Addresses and lengths of a list of contiguous tensors; false when it is not one.
bool listed(PyObject* list, Kind* k, bool first, std::vector<void*>* at, std::vector<long long>* n) {
  if (!PyList_CheckExact(list)) return false;
  const Py_ssize_t count = PyList_GET_SIZE(list);
  at->reserve(count), n->reserve(count);
  for (Py_ssize_t i = 0; i < count; ++i) {
    PyObject* o = PyList_GET_ITEM(list, i);
    if (!is_tensor(o)) return false;
    const Tensor& t = tensor(o);
    if (first && i == 0 && !k->take(t)) return false;
    if (!k->has(t, k->type)) return false;
    at->push_back(ptr(t)), n->push_back(t.numel());
  }
  return count > 0;
}

// Whether no result shares memory with another one, nor with an input other than the tensor
// it replaces.
bool apart(const std::vector<void*>& in, const std::vector<void*>& out,
           const std::vector<long long>& n, int64_t bytes) {
  struct Span {
    uintptr_t from, to;
    size_t i;
    bool operator<(const Span& o) const { return from < o.from; }
  };
  auto span = [&](const std::vector<void*>& at, size_t i) {
    const uintptr_t from = reinterpret_cast<uintptr_t>(at[i]);
    return Span{from, from + (uintptr_t)(n[i] * bytes), i};
  };
  std::vector<Span> outs;
  outs.reserve(out.size());
  for (size_t i = 0; i < out.size(); ++i)
    if (n[i]) outs.push_back(span(out, i));
  if (!std::is_sorted(outs.begin(), outs.end())) std::sort(outs.begin(), outs.end());
  for (size_t k = 1; k < outs.size(); ++k)
    if (outs[k].from < outs[k - 1].to) return false;
  if (&in == &out) return true;
  for (size_t i = 0; i < in.size(); ++i) {
    if (!n[i]) continue;
    const Span x = span(in, i);
    // the results that begin before x's end, from the last one back to x's beginning
    for (auto o = std::lower_bound(outs.begin(), outs.end(), Span{x.to, 0, 0});
         o != outs.begin() && (o - 1)->to > x.from; --o)
      if ((o - 1)->i != i || (o - 1)->from != x.from) return false;
  }
  return true;
}

// grad_norm(grads), or clip_grad_norm(grads, outs, max_norm)
PyObject* clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Kind k;
  std::vector<void*> in, out;
  std::vector<long long> len, out_len;
  double max_norm = 0;
  if ((n != 1 && n != 3) || !listed(a[0], &k, true, &in, &len)) Py_RETURN_NONE;
  if (n == 3) {
    if (!number(a[2], &max_norm)) Py_RETURN_NONE;
    const bool in_place = a[1] == a[0];
    if (!in_place && (!listed(a[1], &k, false, &out, &out_len) || out_len != len)) Py_RETURN_NONE;
    if (!apart(in, in_place ? in : out, len, k.code == B2G_F32 ? 4 : 2)) Py_RETURN_NONE;
    if (in_place) out = in;
  }
  const int count = (int)in.size();
  size_t bytes = 0;
  int rc = b2g_grad_norm_workspace_size(k.code, count, len.data(), &bytes);
  if (rc) return PyLong_FromLong(rc);
  const Tensor norm = k.empty({}, at::kFloat), ws = k.bytes(bytes);
  rc = n == 1 ? b2g_grad_norm(k.code, count, in.data(), len.data(), norm.data_ptr<float>(), ptr(ws),
                              bytes, k.stream)
              : b2g_clip_grad_norm(k.code, count, in.data(), len.data(), (float)max_norm,
                                   out.data(), norm.data_ptr<float>(), ptr(ws), bytes, k.stream);
  return answer(rc, norm);
  END_HANDLE_TH_ERRORS
}

#define FAST(name, fn) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FAST("layer_norm", layer_norm),
    FAST("layer_norm_backward", layer_norm_backward),
    FAST("embedding", embedding),
    FAST("embedding_backward", embedding_backward),
    FAST("linear_cross_entropy", linear_cross_entropy),
    FAST("linear_cross_entropy_backward", linear_cross_entropy_backward),
    FAST("clip", clip),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_train_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__train_binding() { return PyModule_Create(&module); }
