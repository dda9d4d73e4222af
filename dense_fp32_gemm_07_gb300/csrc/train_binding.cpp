// train_binding.cpp -- the tensor calls of train.py and activations.py for plain arguments, in native
// code: contiguous operands of one type on the current device, results that the
// call allocates, the current stream.  Such a call costs the host a few
// microseconds where the same checks and conversions in Python cost 10 to 40,
// which is most of a small call's time.
//
// Each function answers a result as train.py documents it, or the library's error
// code as an int, or None when an argument is not of that plain kind (strided,
// another stream, `out` given, wrong in some way) or torch's dispatcher is watched;
// train.py then goes through its own checks, which serve it or say what is wrong.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/Context.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#include "../../include/b2g_train.h"

namespace {

using at::Tensor;

// Whether somebody looks at the operators that torch dispatches (a mode, a tracer, a function
// transform, a profiler), or wants uninitialised memory filled: both happen in at::empty, which
// Kind::empty goes past.
bool watched() {
  const auto& more = c10::impl::tls_local_dispatch_key_set().included_;
  if (!(more - c10::default_included_set).empty() || at::hasCallbacks()) return true;
  const auto& context = at::globalContext();
  return context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory();
}

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
    return at(t);
  }
  // The device alone.
  bool at(const Tensor& t) {
    device = t.device();
    if (!device.is_cuda() || device.index() != c10::cuda::current_device() || watched()) return false;
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
  // What at::empty ends in on this device, without its dispatch.
  Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::detail::empty_cuda(shape, t, device, c10::nullopt);
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

// Codes and scales in 8 bits: matrices with unit column stride.
struct Eight {
  Tensor q, s;
  int64_t rows, cols;
  long long ldq, lds;

  // New ones, rows on 16-byte boundaries, in one piece of memory: they live together.
  Eight(const Kind& k, int64_t r, int64_t c) : rows(r), cols(c), ldq((c + 15) / 16 * 16), lds((c + 31) / 32) {
    const Tensor all = k.bytes((size_t)(r * (ldq + lds)));
    auto part = [&](at::ScalarType t, int64_t n, int64_t ld, int64_t at) {
      const Tensor x = at::detail::make_tensor<c10::TensorImpl>(
          c10::Storage(all.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
          c10::scalarTypeToTypeMeta(t));
      x.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef{r, n}, at::IntArrayRef{ld, 1}, at);
      return x;
    };
    q = part(at::kFloat8_e4m3fn, c, ldq, 0);
    s = part(at::kFloat8_e8m0fnu, lds, lds, r * ldq);
  }
  Eight(const Tensor& codes, const Tensor& scales) : q(codes), s(scales) {}
  // Whether given ones are on the kind's device and fit each other.
  bool take(const Kind& k) {
    if (q.scalar_type() != at::kFloat8_e4m3fn || s.scalar_type() != at::kFloat8_e8m0fnu ||
        q.device() != k.device || s.device() != k.device || q.dim() != 2 || s.dim() != 2 ||
        !s.is_contiguous())
      return false;
    rows = q.size(0), cols = q.size(1), ldq = q.stride(0), lds = s.size(1);
    return rows > 0 && cols > 1 && q.stride(1) == 1 && ldq >= cols && s.size(0) == rows &&
           lds == (cols + 31) / 32;
  }
};

PyObject* pair(const Eight& e) {
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, wrap(e.q));
  PyTuple_SET_ITEM(t, 1, wrap(e.s));
  return t;
}

// quantize_8bit(x)
PyObject* quantize_8bit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 1 || !is_tensor(a[0])) Py_RETURN_NONE;
  const Tensor& x = tensor(a[0]);
  Kind k;
  if (!k.take(x) || !k.matrix(x)) Py_RETURN_NONE;
  const int64_t r = x.size(0), c = x.size(1);
  if (!small(c) || c == 0) Py_RETURN_NONE;
  const Eight e(k, r, c);
  const int rc = b2g_quantize8(k.code, r, (int)c, ptr(x), c, ptr(e.q), e.ldq, ptr(e.s), e.lds, k.stream);
  return rc ? PyLong_FromLong(rc) : pair(e);
  END_HANDLE_TH_ERRORS
}

// dequantize_8bit(codes, scales, dtype or None)
PyObject* dequantize_8bit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3 || !is_tensor(a[0]) || !is_tensor(a[1])) Py_RETURN_NONE;
  at::ScalarType type = at::kBFloat16;
  if (a[2] != Py_None) {
    if (!THPDtype_Check(a[2])) Py_RETURN_NONE;
    type = reinterpret_cast<THPDtype*>(a[2])->scalar_type;
    if (type != at::kFloat && type != at::kBFloat16) Py_RETURN_NONE;
  }
  Eight e(tensor(a[0]), tensor(a[1]));
  Kind k;
  if (!k.at(e.q) || !e.take(k) || !small(e.cols)) Py_RETURN_NONE;
  const Tensor y = k.empty({e.rows, e.cols}, type);
  const int rc = b2g_dequantize8(type == at::kFloat ? B2G_F32 : B2G_BF16, e.rows, (int)e.cols, ptr(e.q),
                                 e.ldq, ptr(e.s), e.lds, ptr(y), e.cols, k.stream);
  return answer(rc, y);
  END_HANDLE_TH_ERRORS
}

// rms_norm(x, weight, residual, eps), or rms_norm_8bit(.., with_y, keep_total)
PyObject* rms(PyObject* const* a, Py_ssize_t n, bool eight) {
  double eps;
  if (n != (eight ? 6 : 4) || !is_tensor(a[0]) || !is_tensor_or_none(a[1]) ||
      !is_tensor_or_none(a[2]) || !number(a[3], &eps) ||
      (eight && (!PyBool_Check(a[4]) || !PyBool_Check(a[5]))))
    Py_RETURN_NONE;
  const Tensor &x = tensor(a[0]), &w = tensor(a[1]), &res = tensor(a[2]);
  Kind k;
  if (!k.take(x) || !k.matrix(x)) Py_RETURN_NONE;
  const int64_t r = x.size(0), c = x.size(1);
  if (!small(c) || c == 0 || (w.defined() && !k.vector(w, k.type, c)) ||
      (res.defined() && (!k.matrix(res) || res.sizes() != x.sizes())))
    Py_RETURN_NONE;
  const bool with_y = !eight || a[4] == Py_True, keep = eight && a[5] == Py_True;
  const Tensor y = with_y ? k.empty({r, c}) : Tensor(), total = res.defined() ? k.empty({r, c}) : x,
               rstd = k.empty({r}, at::kFloat);
  const Eight none{Tensor(), Tensor()};
  const Eight y8 = eight ? Eight(k, r, c) : none, t8 = keep ? Eight(k, r, c) : none;
  auto at = [](const Tensor& t) { return t.defined() ? ptr(t) : nullptr; };
  const int rc = b2g_rmsnorm(k.code, r, (int)c, ptr(x), c, at(res), c, at(w), (float)eps,
                             res.defined() ? ptr(total) : nullptr, c, at(y), c, at(y8.q), eight ? y8.ldq : 0,
                             at(y8.s), eight ? y8.lds : 0, at(t8.q), keep ? t8.ldq : 0, at(t8.s),
                             keep ? t8.lds : 0, rstd.data_ptr<float>(), k.stream);
  if (!eight) return answer(rc, y, total, rstd);
  if (rc) return PyLong_FromLong(rc);
  PyObject* out = PyTuple_New(5);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, wrap(y));
  PyTuple_SET_ITEM(out, 1, wrap(total));
  PyTuple_SET_ITEM(out, 2, wrap(rstd));
  PyObject *p = pair(y8), *q = keep ? pair(t8) : Py_NewRef(Py_None);
  PyTuple_SET_ITEM(out, 3, p);
  PyTuple_SET_ITEM(out, 4, q);
  if (p && q) return out;
  Py_DECREF(out);
  return nullptr;
}
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return rms(a, n, false);
  END_HANDLE_TH_ERRORS
}
PyObject* rms_norm_8bit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return rms(a, n, true);
  END_HANDLE_TH_ERRORS
}

// rms_norm_backward(dy, total or (codes, scales), weight, rstd, dtotal)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !is_tensor(a[0]) || !is_tensor_or_none(a[2]) || !is_tensor(a[3]) ||
      !is_tensor_or_none(a[4]))
    Py_RETURN_NONE;
  const Tensor &dy = tensor(a[0]), &w = tensor(a[2]), &rstd = tensor(a[3]), &dt = tensor(a[4]);
  Kind k;
  if (!k.take(dy) || !k.matrix(dy)) Py_RETURN_NONE;
  const int64_t r = dy.size(0), c = dy.size(1);
  const void *x, *scales = nullptr;
  long long ldx = c, lds = 0;
  if (is_tensor(a[1])) {
    const Tensor& t = tensor(a[1]);
    if (!k.matrix(t) || t.sizes() != dy.sizes()) Py_RETURN_NONE;
    x = ptr(t);
  } else {
    if (!PyTuple_CheckExact(a[1]) || PyTuple_GET_SIZE(a[1]) != 2 ||
        !is_tensor(PyTuple_GET_ITEM(a[1], 0)) || !is_tensor(PyTuple_GET_ITEM(a[1], 1)))
      Py_RETURN_NONE;
    Eight e(tensor(PyTuple_GET_ITEM(a[1], 0)), tensor(PyTuple_GET_ITEM(a[1], 1)));
    if (!e.take(k) || e.rows != r || e.cols != c) Py_RETURN_NONE;
    x = ptr(e.q), ldx = e.ldq, scales = ptr(e.s), lds = e.lds;
  }
  if (!small(c) || c == 0 || (w.defined() && !k.vector(w, k.type, c)) || !k.vector(rstd, at::kFloat, r) ||
      (dt.defined() && (!k.matrix(dt) || dt.sizes() != dy.sizes())))
    Py_RETURN_NONE;
  size_t bytes = 0;
  int rc = w.defined() ? b2g_rmsnorm_backward_workspace_size(k.code, r, (int)c, &bytes) : 0;
  if (rc) return PyLong_FromLong(rc);
  const Tensor dx = k.empty({r, c}), dw = w.defined() ? k.empty({c}) : Tensor(), ws = k.bytes(bytes);
  rc = b2g_rmsnorm_backward(k.code, r, (int)c, ptr(dy), c, x, ldx, scales, lds,
                            w.defined() ? ptr(w) : nullptr, rstd.data_ptr<float>(),
                            dt.defined() ? ptr(dt) : nullptr, c, ptr(dx), c,
                            dw.defined() ? ptr(dw) : nullptr, ptr(ws), bytes, k.stream);
  return answer(rc, dx, dw);
  END_HANDLE_TH_ERRORS
}

// Whether a contiguous tensor and `bytes` from `at` on have nothing in common.
bool clear_of(const Tensor& t, const void* at, int64_t bytes) {
  const char *a = static_cast<const char*>(ptr(t)), *b = static_cast<const char*>(at);
  return a + t.nbytes() <= b || b + bytes <= a;
}

// linear_weight_grad_8bit(dy, codes, scales, dw, accumulate)
PyObject* linear_weight_grad_8bit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !is_tensor(a[0]) || !is_tensor(a[1]) || !is_tensor(a[2]) || !is_tensor_or_none(a[3]) ||
      !PyBool_Check(a[4]))
    Py_RETURN_NONE;
  const Tensor &dy = tensor(a[0]), &given = tensor(a[3]);
  const bool accumulate = a[4] == Py_True;
  Eight e(tensor(a[1]), tensor(a[2]));
  Kind k;
  if (!k.take(dy) || !k.matrix(dy) || !e.take(k) || e.rows != dy.size(0)) Py_RETURN_NONE;
  const int64_t t = e.rows, o = dy.size(1);
  if (!small(t) || !small(o) || !small(e.cols)) Py_RETURN_NONE;
  if (given.defined()) {
    if (!k.matrix(given) || given.size(0) != o || given.size(1) != e.cols ||
        !clear_of(given, ptr(dy), dy.nbytes()) || !clear_of(given, ptr(e.q), e.rows * e.ldq) ||
        !clear_of(given, ptr(e.s), e.rows * e.lds))
      Py_RETURN_NONE;
  } else if (accumulate) {
    Py_RETURN_NONE;
  }
  size_t bytes = 0;
  int rc = b2g_linear_dweight8_workspace_size_ex(k.code, (int)t, (int)o, (int)e.cols, ptr(dy), ld(o), ptr(e.q),
                                                 e.ldq, &bytes);
  if (rc) return PyLong_FromLong(rc);
  const Tensor dw = given.defined() ? given : k.empty({o, e.cols}), ws = k.bytes(bytes);
  rc = b2g_linear_dweight8(k.code, (int)t, (int)o, (int)e.cols, ptr(dy), ld(o), ptr(e.q), e.ldq, ptr(e.s),
                           e.lds, accumulate, ptr(dw), e.cols, ptr(ws), bytes, k.stream);
  if (rc || !given.defined()) return answer(rc, dw);
  Py_INCREF(a[3]);
  return a[3];
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
    FAST("quantize_8bit", quantize_8bit),
    FAST("dequantize_8bit", dequantize_8bit),
    FAST("rms_norm", rms_norm),
    FAST("rms_norm_8bit", rms_norm_8bit),
    FAST("rms_norm_backward", rms_norm_backward),
    FAST("linear_weight_grad_8bit", linear_weight_grad_8bit),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_train_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__train_binding() { return PyModule_Create(&module); }
