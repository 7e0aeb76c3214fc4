// CPython module memory_bounded_linear_gb300._native: the feed-forward, clipping, normalisation, embedding
// and sampling entry points on torch tensors.  Checks of arguments, allocation of results, the current stream, the C call.
//
// These operators are called once per layer and decoded token, where kernels run for 5 to 25
// microseconds; the same marshalling in Python took 15 us of every call, here about 2.
// A C status other than LCE_OK is returned as an int for the caller to raise; bad tensors raise
// ValueError or TypeError here.  No exception leaves an entry point.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <sstream>
#include <string>
#include <vector>

#include "lce.h"

namespace {

struct Refused {
  PyObject* type;
  std::string what;
};
template <typename... A>
[[noreturn]] void refuse(PyObject* type, const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused{type, s.str()};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, " must be a tensor");
  return THPVariable_Unpack(o);
}

const char* dtype_name(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    default: return toString(t.scalar_type());
  }
}

lce_dtype_t dtype_of(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return LCE_BF16;
  if (t.scalar_type() == at::kFloat) return LCE_F32;
  refuse(PyExc_TypeError, what, " must be bfloat16 or float32, got ", dtype_name(t));
}

void same_kind(const at::Tensor& t, const char* name, const at::Tensor& x) {
  if (t.scalar_type() != x.scalar_type())
    refuse(PyExc_TypeError, name, " must have the dtype of X (", dtype_name(x), "), got ", dtype_name(t));
  if (t.device() != x.device())
    refuse(PyExc_ValueError, name, " must be a CUDA tensor on the device of X");
}

// A matrix with unit column stride; returns its row stride.
int64_t rows(const at::Tensor& t, const char* name, int64_t n, int64_t width, const at::Tensor& x) {
  same_kind(t, name, x);
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != width)
    refuse(PyExc_ValueError, "expected ", name, " [", n, ", ", width, "], got ", t.sizes());
  if (t.is_contiguous()) return width;
  if ((width > 1 && t.stride(1) != 1) || (n > 1 && t.stride(0) < width))
    refuse(PyExc_ValueError, name, " must have contiguous, non-overlapping rows (strides ",
           t.strides(), ")");
  return n > 1 ? t.stride(0) : width;
}

void dense(const at::Tensor& t, const char* name, at::IntArrayRef shape, const at::Tensor& x) {
  same_kind(t, name, x);
  if (t.sizes() != shape) refuse(PyExc_ValueError, "expected ", name, " ", shape, ", got ", t.sizes());
  if (!t.is_contiguous()) refuse(PyExc_ValueError, name, " must be contiguous");
}

// Sizes of X [N, d] against W [width, d].
struct Sizes {
  int64_t N, d, width;
  lce_dtype_t dt;
};
Sizes sizes(const at::Tensor& x, const at::Tensor& w) {
  if (!x.is_cuda()) refuse(PyExc_ValueError, "X must be a CUDA tensor");
  if (x.dim() != 2 || w.dim() != 2 || x.size(1) != w.size(1))
    refuse(PyExc_ValueError, "expected X [N, d] and W [width, d], got ", x.sizes(), " and ", w.sizes());
  return Sizes{x.size(0), x.size(1), w.size(0), dtype_of(x, "X and W")};
}

// The caller's workspace, or a new one of `size` bytes.
at::Tensor workspace(PyObject* given, size_t size, const at::Tensor& x) {
  if (given == Py_None)
    return at::empty({static_cast<int64_t>(size)}, x.options().dtype(at::kByte));
  const at::Tensor& t = tensor(given, "workspace");
  if (t.device() != x.device())
    refuse(PyExc_ValueError, "workspace must be on ", x.device(), ", got ", t.device());
  if (t.scalar_type() != at::kByte || !t.is_contiguous())
    refuse(PyExc_ValueError, "workspace must be a contiguous uint8 tensor");
  return t;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
void* stream_of(const at::Tensor& x) {
  return c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
}
PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* status(lce_status_t st) { return PyLong_FromLong(st); }

// Tells autograd that a caller's tensor is written: a backward pass that saved its old values then
// raises instead of using the new ones.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

template <typename... T>
PyObject* tuple_of(const T&... t) {
  PyObject* items[] = {wrap(t)...};
  constexpr int n = sizeof...(T);
  for (int i = 0; i < n; ++i)
    if (!items[i]) {
      for (int j = 0; j < n; ++j) Py_XDECREF(items[j]);
      return nullptr;
    }
  PyObject* r = PyTuple_New(n);
  for (int i = 0; i < n; ++i) {
    if (r) PyTuple_SET_ITEM(r, i, items[i]);
    else Py_DECREF(items[i]);
  }
  return r;
}

at::Tensor optional(PyObject* o, const char* name) {
  return o == Py_None ? at::Tensor() : tensor(o, name);
}

lce_activation_t activation(PyObject* o) {
  return static_cast<lce_activation_t>(PyLong_AsLong(o));
}

// (X, W, bias, residual, activation, out, workspace) -> (Y, workspace) or a status
PyObject* linear_forward(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "X"), &w = tensor(a[1], "W");
  const Sizes s = sizes(x, w);
  const int64_t ldx = rows(x, "X", s.N, s.d, x);
  dense(w, "W", {s.width, s.d}, x);
  const at::Tensor bias = optional(a[2], "bias"), res = optional(a[3], "residual");
  if (bias.defined()) dense(bias, "bias", {s.width}, x);
  const int64_t ldr = res.defined() ? rows(res, "residual", s.N, s.width, x) : 0;
  const lce_activation_t act = activation(a[4]);
  at::Tensor out = optional(a[5], "out");
  const int64_t ldy = out.defined() ? rows(out, "out", s.N, s.width, x) : s.width;
  const size_t need = lce_linear_workspace_size(s.N, s.d, s.width, act, 0, s.dt);
  if (need == 0) return status(LCE_ERR_UNSUPPORTED_SHAPE);
  const c10::cuda::CUDAGuard guard(x.device());
  const at::Tensor ws = workspace(a[6], need, x);
  if (out.defined()) written(out);
  else out = at::empty({s.N, s.width}, x.options());
  const lce_status_t st =
      lce_linear_forward(ptr(x), ldx, ptr(w), ptr(bias), ptr(res), ldr, s.N, s.d, s.width, act, s.dt,
                         ptr(out), ldy, ptr(ws), ws.numel(), stream_of(x));
  return st == LCE_OK ? tuple_of(out, ws) : status(st);
}

// (X, W, bias, dY, activation, want_dx, want_dw, workspace) -> (dX, dW, dbias, workspace) or a status
PyObject* linear_backward(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "X"), &w = tensor(a[1], "W"), &dy = tensor(a[3], "dY");
  const Sizes s = sizes(x, w);
  const int64_t ldx = rows(x, "X", s.N, s.d, x);
  dense(w, "W", {s.width, s.d}, x);
  const at::Tensor bias = optional(a[2], "bias");
  if (bias.defined()) dense(bias, "bias", {s.width}, x);
  const int64_t ldy = rows(dy, "dY", s.N, s.width, x);
  const lce_activation_t act = activation(a[4]);
  const bool want_dx = a[5] == Py_True, want_dw = a[6] == Py_True;
  const size_t need = lce_linear_workspace_size(s.N, s.d, s.width, act, 1, s.dt);
  if (need == 0) return status(LCE_ERR_UNSUPPORTED_SHAPE);
  const c10::cuda::CUDAGuard guard(x.device());
  const at::Tensor ws = workspace(a[7], need, x);
  at::Tensor dx, dw, db;
  if (want_dx) dx = at::empty({s.N, s.d}, x.options());
  if (want_dw) dw = at::empty({s.width, s.d}, x.options());
  if (want_dw && bias.defined()) db = at::empty({s.width}, x.options());
  const lce_status_t st =
      lce_linear_backward(ptr(x), ldx, ptr(w), ptr(bias), ptr(dy), ldy, s.N, s.d, s.width, act, s.dt,
                          ptr(dx), ptr(dw), ptr(db), ptr(ws), ws.numel(), stream_of(x));
  return st == LCE_OK ? tuple_of(dx, dw, db, ws) : status(st);
}

// (X, Wg, Wu, activation, out, workspace) -> (H, workspace) or a status
PyObject* gated_forward(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "X"), &wg = tensor(a[1], "Wg"), &wu = tensor(a[2], "Wu");
  const Sizes s = sizes(x, wg);
  const int64_t ldx = rows(x, "X", s.N, s.d, x);
  dense(wg, "Wg", {s.width, s.d}, x);
  dense(wu, "Wu", {s.width, s.d}, x);
  const lce_activation_t act = activation(a[3]);
  at::Tensor out = optional(a[4], "out");
  const int64_t ldh = out.defined() ? rows(out, "out", s.N, s.width, x) : s.width;
  const size_t need = lce_gated_workspace_size(s.N, s.d, s.width, 0, s.dt);
  if (need == 0) return status(LCE_ERR_UNSUPPORTED_SHAPE);
  const c10::cuda::CUDAGuard guard(x.device());
  const at::Tensor ws = workspace(a[5], need, x);
  if (out.defined()) written(out);
  else out = at::empty({s.N, s.width}, x.options());
  const lce_status_t st =
      lce_gated_forward(ptr(x), ldx, ptr(wg), ptr(wu), s.N, s.d, s.width, act, s.dt, ptr(out), ldh,
                        ptr(ws), ws.numel(), stream_of(x));
  return st == LCE_OK ? tuple_of(out, ws) : status(st);
}

// (X, Wg, Wu, dH, activation, want_dx, want_dw, workspace) -> (dX, dWg, dWu, workspace) or a status
PyObject* gated_backward(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "X"), &wg = tensor(a[1], "Wg"), &wu = tensor(a[2], "Wu"),
                   &dh = tensor(a[3], "dH");
  const Sizes s = sizes(x, wg);
  const int64_t ldx = rows(x, "X", s.N, s.d, x);
  dense(wg, "Wg", {s.width, s.d}, x);
  dense(wu, "Wu", {s.width, s.d}, x);
  const int64_t ldh = rows(dh, "dH", s.N, s.width, x);
  const lce_activation_t act = activation(a[4]);
  const bool want_dx = a[5] == Py_True, want_dw = a[6] == Py_True;
  const size_t need = lce_gated_workspace_size(s.N, s.d, s.width, 1, s.dt);
  if (need == 0) return status(LCE_ERR_UNSUPPORTED_SHAPE);
  const c10::cuda::CUDAGuard guard(x.device());
  const at::Tensor ws = workspace(a[7], need, x);
  at::Tensor dx, dwg, dwu;
  if (want_dx) dx = at::empty({s.N, s.d}, x.options());
  if (want_dw) {
    dwg = at::empty({s.width, s.d}, x.options());
    dwu = at::empty({s.width, s.d}, x.options());
  }
  const lce_status_t st =
      lce_gated_backward(ptr(x), ldx, ptr(wg), ptr(wu), ptr(dh), ldh, s.N, s.d, s.width, act, s.dt,
                         ptr(dx), ptr(dwg), ptr(dwu), ptr(ws), ws.numel(), stream_of(x));
  return st == LCE_OK ? tuple_of(dx, dwg, dwu, ws) : status(st);
}

// Refuses outputs that share memory with another output, or with an input that is not the same array:
// blocks that run at the same time would read values that others have scaled already.  Inputs may
// share memory with one another where nothing is written to it.
void check_overlap(const std::vector<const void*>& in, const std::vector<void*>& out,
                   const std::vector<int64_t>& bytes) {
  struct Span {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Span> spans;
  spans.reserve(2 * in.size());
  auto add = [&](const void* p, int64_t n, bool written) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    if (n > 0) spans.push_back(Span{b, b + static_cast<uintptr_t>(n), written});
  };
  for (size_t i = 0; i < in.size(); ++i) {
    const void* o = out.empty() ? in[i] : out[i];
    add(o, bytes[i], true);
    if (o != in[i]) add(in[i], bytes[i], false);
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t read = 0, written = 0;  // ends of what came so far
  for (const Span& s : spans) {
    if (s.begin < written || (s.written && s.begin < read))
      refuse(PyExc_ValueError, "an array that is written overlaps another one of the call");
    uintptr_t& end = s.written ? written : read;
    end = std::max(end, s.end);
  }
}

// (gradients, out or None, norm, max_norm or None, workspace) -> (total, workspace) or a status;
// without max_norm the norm alone.
PyObject* clip(PyObject* const* a) {
  struct Held {  // a list or tuple of the sequence, released on every way out
    PyObject* o;
    explicit Held(PyObject* s) : o(PySequence_Fast(s, "expected a sequence of tensors")) {
      if (!o) throw python_error();
    }
    ~Held() { Py_DECREF(o); }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(o); }
    PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(o, i); }
  };
  const Held grads(a[0]);
  const Py_ssize_t n = grads.size();
  if (n == 0) refuse(PyExc_ValueError, "no gradients");
  const at::Tensor first = tensor(grads.at(0), "a gradient");
  if (!first.is_cuda()) refuse(PyExc_ValueError, "gradients must be CUDA tensors");
  std::vector<const void*> in(n);
  std::vector<void*> out;
  std::vector<int64_t> numel(n), bytes(n);
  std::vector<int32_t> dt(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor& t = tensor(grads.at(i), "a gradient");
    if (!t.is_cuda()) refuse(PyExc_ValueError, "gradients must be CUDA tensors");
    if (t.device() != first.device()) refuse(PyExc_ValueError, "gradients must be on one device");
    dt[i] = dtype_of(t, "gradients");
    if (!t.is_non_overlapping_and_dense())
      refuse(PyExc_ValueError, "gradients must be dense (strides ", t.strides(), " of ", t.sizes(), ")");
    in[i] = t.data_ptr();
    numel[i] = t.numel();
    bytes[i] = t.nbytes();
  }
  if (a[1] != Py_None) {
    const Held outs(a[1]);
    if (outs.size() != n) refuse(PyExc_ValueError, n, " gradients and ", outs.size(), " outputs");
    out.resize(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor &t = tensor(grads.at(i), "a gradient"), &o = tensor(outs.at(i), "an output");
      if (o.scalar_type() != t.scalar_type() || o.device() != t.device() || o.sizes() != t.sizes() ||
          !((t.is_contiguous() && o.is_contiguous()) || o.strides() == t.strides()))
        refuse(PyExc_ValueError, "each output must have its gradient's dtype, shape, strides and device");
      out[i] = o.data_ptr();
    }
  }
  if (a[3] != Py_None) check_overlap(in, out, bytes);
  const lce_norm_t norm = static_cast<lce_norm_t>(PyLong_AsLong(a[2]));
  const size_t need = lce_grad_norm_workspace_size(n);
  if (need == 0) return status(LCE_ERR_UNSUPPORTED_SHAPE);
  const c10::cuda::CUDAGuard guard(first.device());
  const at::Tensor ws = workspace(a[4], need, first);
  const at::Tensor total = at::empty({}, first.options().dtype(at::kFloat));
  float* tp = static_cast<float*>(total.data_ptr());
  if (a[3] != Py_None) {
    const Held written_to(a[1] == Py_None ? a[0] : a[1]);
    for (Py_ssize_t i = 0; i < n; ++i) written(tensor(written_to.at(i), "an output"));
  }
  const lce_status_t st =
      a[3] == Py_None
          ? lce_grad_norm(in.data(), numel.data(), dt.data(), n, norm, tp, ptr(ws), ws.numel(),
                          stream_of(first))
          : lce_clip_grad_norm(in.data(), out.empty() ? nullptr : out.data(), numel.data(), dt.data(),
                               n, norm, static_cast<float>(PyFloat_AsDouble(a[3])), tp, ptr(ws),
                               ws.numel(), stream_of(first));
  return st == LCE_OK ? tuple_of(total, ws) : status(st);
}

// The bytes that a matrix of rows takes.
struct Span {
  uintptr_t begin, end;
  size_t rows, stride, width;  // bytes of a row's step and of a row
};
Span span_of(const at::Tensor& t) {
  const size_t e = t.element_size();
  const size_t width = t.dim() ? t.size(-1) * e : e;
  const size_t n = t.dim() == 2 ? t.size(0) : 1;
  const size_t stride = t.dim() == 2 && n > 1 ? t.stride(0) * e : width;
  const uintptr_t b = reinterpret_cast<uintptr_t>(t.data_ptr());
  return Span{b, t.numel() ? b + (n - 1) * stride + width : b, n, stride, width};
}
// Refuses an output that shares elements with another array of the call.  Column ranges of one wider array
// do not, nor does a single row between the rows of one.
void apart(const at::Tensor& out, const char* name, const at::Tensor& in, const char* other) {
  if (!in.defined()) return;
  const Span a = span_of(out), b = span_of(in);
  if (a.begin >= b.end || b.begin >= a.end) return;
  const size_t stride = a.rows == 1 ? b.stride : b.rows == 1 || a.stride == b.stride ? a.stride : 0;
  if (stride > 0) {
    const size_t off = (b.begin >= a.begin ? b.begin - a.begin : stride - (a.begin - b.begin) % stride) % stride;
    if (off >= a.width && off + b.width <= stride) return;
  }
  refuse(PyExc_ValueError, name, " shares memory with ", other);
}

// A vector of n elements of the dtype of X, or none.
at::Tensor vector(PyObject* o, const char* name, int64_t n, const at::Tensor& x) {
  const at::Tensor t = optional(o, name);
  if (t.defined()) dense(t, name, {n}, x);
  return t;
}
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, name, " must be a number");
  }
  return v;
}
int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, name, " must be an integer of 64 bits");
  }
  return v;
}
// X [N, d], and what the matrices of a normalisation share.
const at::Tensor& matrix(PyObject* o, const char* name) {
  const at::Tensor& x = tensor(o, name);
  if (!x.is_cuda()) refuse(PyExc_ValueError, name, " must be a CUDA tensor");
  if (x.dim() != 2) refuse(PyExc_ValueError, "expected ", name, " of two dimensions, got ", x.sizes());
  return x;
}

// (X, weight, bias, eps, out) -> Y or a status
PyObject* layer_norm_forward(PyObject* const* a) {
  const at::Tensor& x = matrix(a[0], "X");
  const lce_dtype_t dt = dtype_of(x, "X");
  const int64_t N = x.size(0), d = x.size(1);
  const int64_t ldx = rows(x, "X", N, d, x);
  const at::Tensor w = vector(a[1], "weight", d, x), b = vector(a[2], "bias", d, x);
  const float eps = static_cast<float>(number(a[3], "eps"));
  at::Tensor out = optional(a[4], "out");
  const int64_t ldy = out.defined() ? rows(out, "out", N, d, x) : d;
  if (out.defined()) {
    if (out.data_ptr() != x.data_ptr() || (ldx != ldy && N > 1)) apart(out, "out", x, "X");
    apart(out, "out", w, "weight");
    apart(out, "out", b, "bias");
  }
  const c10::cuda::CUDAGuard guard(x.device());
  if (out.defined()) written(out);
  else out = at::empty({N, d}, x.options());
  const lce_status_t st = lce_layer_norm_forward(ptr(x), ldx, ptr(w), ptr(b), N, d, eps, dt, ptr(out), ldy,
                                                 stream_of(x));
  return st == LCE_OK ? wrap(out) : status(st);
}

// (X, weight, bias, dY, eps, want_dx, want_dw, workspace) -> (dX, dweight, dbias, workspace) or a status
PyObject* layer_norm_backward(PyObject* const* a) {
  const at::Tensor &x = matrix(a[0], "X"), &dy = tensor(a[3], "dY");
  const lce_dtype_t dt = dtype_of(x, "X");
  const int64_t N = x.size(0), d = x.size(1);
  const int64_t ldx = rows(x, "X", N, d, x), ldy = rows(dy, "dY", N, d, x);
  const at::Tensor w = vector(a[1], "weight", d, x), b = vector(a[2], "bias", d, x);
  const float eps = static_cast<float>(number(a[4], "eps"));
  const bool want_dx = a[5] == Py_True, want_dw = a[6] == Py_True;
  const size_t need = lce_layer_norm_workspace_size(N, d, dt);
  if (need == 0) return status(LCE_ERR_UNSUPPORTED_SHAPE);
  const c10::cuda::CUDAGuard guard(x.device());
  const at::Tensor ws = workspace(a[7], need, x);
  at::Tensor dx, dw, db;
  if (want_dx) dx = at::empty({N, d}, x.options());
  if (want_dw && w.defined()) dw = at::empty({d}, x.options());
  if (want_dw && b.defined()) db = at::empty({d}, x.options());
  const lce_status_t st =
      lce_layer_norm_backward(ptr(x), ldx, ptr(w), ptr(dy), ldy, N, d, eps, dt, ptr(dx), ptr(dw), ptr(db),
                              ptr(ws), ws.numel(), stream_of(x));
  return st == LCE_OK ? tuple_of(dx, dw, db, ws) : status(st);
}

// int64 [N] on the device of `like`.
const at::Tensor& token_list(PyObject* o, const at::Tensor& like, const char* other) {
  const at::Tensor& t = tensor(o, "tokens");
  if (t.device() != like.device()) refuse(PyExc_ValueError, "tokens must be a CUDA tensor on the device of ", other);
  if (t.scalar_type() != at::kLong) refuse(PyExc_TypeError, "tokens must be int64, got ", toString(t.scalar_type()));
  if (t.dim() != 1 || !t.is_contiguous())
    refuse(PyExc_ValueError, "tokens must be contiguous and of one dimension, got ", t.sizes());
  return t;
}

// (tokens, table, scale, ignore_index, out, workspace) -> (Y, workspace) or a status
PyObject* embedding_forward(PyObject* const* a) {
  const at::Tensor& table = matrix(a[1], "table");
  const lce_dtype_t dt = dtype_of(table, "table");
  const at::Tensor& tokens = token_list(a[0], table, "table");
  const int64_t N = tokens.size(0), V = table.size(0), d = table.size(1);
  if (!table.is_contiguous()) refuse(PyExc_ValueError, "table must be contiguous");
  const float scale = static_cast<float>(number(a[2], "scale"));
  const int64_t ignore = integer(a[3], "ignore_index");
  at::Tensor out = optional(a[4], "out");
  if (out.defined() && out.scalar_type() != table.scalar_type())
    refuse(PyExc_TypeError, "out must have the dtype of table (", dtype_name(table), "), got ", dtype_name(out));
  const int64_t ldy = out.defined() ? rows(out, "out", N, d, table) : d;
  if (out.defined()) {
    apart(out, "out", table, "table");
    apart(out, "out", tokens, "tokens");
  }
  const size_t need = lce_embedding_workspace_size(N, d, V, 0);
  if (need == 0) return status(LCE_ERR_UNSUPPORTED_SHAPE);
  const c10::cuda::CUDAGuard guard(table.device());
  const at::Tensor ws = workspace(a[5], need, table);
  if (out.defined()) written(out);
  else out = at::empty({N, d}, table.options());
  const lce_status_t st = lce_embedding_forward(static_cast<const int64_t*>(ptr(tokens)), ptr(table), N, d, V,
                                                scale, ignore, dt, ptr(out), ldy, ptr(ws), ws.numel(),
                                                stream_of(table));
  return st == LCE_OK ? tuple_of(out, ws) : status(st);
}

// (tokens, dY, V, scale, ignore_index, float32 gradient, out, accumulate, workspace) -> (dtable, workspace) or a
// status
PyObject* embedding_backward(PyObject* const* a) {
  const at::Tensor& dy = matrix(a[1], "dY");
  const lce_dtype_t dt = dtype_of(dy, "dY");
  const at::Tensor& tokens = token_list(a[0], dy, "dY");
  const int64_t N = dy.size(0), d = dy.size(1), V = integer(a[2], "V");
  if (tokens.size(0) != N) refuse(PyExc_ValueError, "expected tokens [", N, "], got ", tokens.sizes());
  const int64_t ldy = rows(dy, "dY", N, d, dy);
  const float scale = static_cast<float>(number(a[3], "scale"));
  const int64_t ignore = integer(a[4], "ignore_index");
  at::Tensor out = optional(a[6], "out");
  const bool accumulate = a[7] == Py_True;
  lce_dtype_t gt = a[5] == Py_True ? LCE_F32 : dt;
  if (accumulate && !out.defined()) refuse(PyExc_ValueError, "accumulate needs out");
  if (out.defined()) {
    if (out.device() != dy.device()) refuse(PyExc_ValueError, "out must be a CUDA tensor on the device of dY");
    gt = dtype_of(out, "out");
    if (gt != dt && gt != LCE_F32) refuse(PyExc_TypeError, "out must be float32 or have the dtype of dY");
    if (out.dim() != 2 || out.size(0) != V || out.size(1) != d || !out.is_contiguous())
      refuse(PyExc_ValueError, "expected a contiguous out [", V, ", ", d, "], got ", out.sizes());
    apart(out, "out", dy, "dY");
    apart(out, "out", tokens, "tokens");
  }
  const size_t need = lce_embedding_workspace_size(N, d, V, 1);
  if (need == 0) return status(LCE_ERR_UNSUPPORTED_SHAPE);
  const c10::cuda::CUDAGuard guard(dy.device());
  const at::Tensor ws = workspace(a[8], need, dy);
  if (out.defined()) written(out);
  else out = at::empty({V, d}, dy.options().dtype(gt == LCE_F32 ? at::kFloat : at::kBFloat16));
  const lce_status_t st =
      lce_embedding_backward(static_cast<const int64_t*>(ptr(tokens)), ptr(dy), ldy, N, d, V, scale, ignore, dt, gt,
                             accumulate, ptr(out), ptr(ws), ws.numel(), stream_of(dy));
  return st == LCE_OK ? tuple_of(out, ws) : status(st);
}

// One value for all rows, or a tensor of one a row.
const void* setting(PyObject* o, const char* name, at::ScalarType type, int64_t B, const at::Tensor& x) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.device() != x.device()) refuse(PyExc_ValueError, name, " must be a number or on the device of logits");
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, name, " must be a number or ", toString(type), ", got ", toString(t.scalar_type()));
  if (t.dim() != 1 || t.size(0) != B || !t.is_contiguous())
    refuse(PyExc_ValueError, name, " must be a number or a contiguous tensor [", B, "], got ", t.sizes());
  return t.data_ptr();
}
float share(PyObject* o, const char* name, double most) {
  const double v = number(o, name);
  if (!(v >= 0.0 && v <= most))
    refuse(PyExc_ValueError, name, most == 1.0 ? " must be from 0 to 1, got " : " must be at least 0, got ", v);
  return static_cast<float>(v);
}

// (logits, uniform, temperature, top_k, top_p, min_p, tokens or None, logprobs or None) -> (tokens, logprobs) or a
// status
PyObject* sample(PyObject* const* a) {
  const at::Tensor& x = matrix(a[0], "logits");
  const lce_dtype_t dt = dtype_of(x, "logits");
  const int64_t B = x.size(0), V = x.size(1);
  const int64_t ld = rows(x, "logits", B, V, x);
  if (!THPVariable_Check(a[1])) refuse(PyExc_TypeError, "uniform must be a tensor");
  const void* u = setting(a[1], "uniform", at::kFloat, B, x);
  lce_sampling_t set{};
  set.temperatures = static_cast<const float*>(setting(a[2], "temperature", at::kFloat, B, x));
  if (!THPVariable_Check(a[2])) set.temperature = share(a[2], "temperature", HUGE_VAL);
  set.top_ks = static_cast<const int32_t*>(setting(a[3], "top_k", at::kInt, B, x));
  if (!THPVariable_Check(a[3])) {
    const int64_t k = integer(a[3], "top_k");
    if (k < 0) refuse(PyExc_ValueError, "top_k must be at least 0, got ", k);
    set.top_k = static_cast<int32_t>(std::min<int64_t>(k, INT32_MAX));
  }
  set.top_ps = static_cast<const float*>(setting(a[4], "top_p", at::kFloat, B, x));
  if (!THPVariable_Check(a[4])) set.top_p = share(a[4], "top_p", 1.0);
  set.min_ps = static_cast<const float*>(setting(a[5], "min_p", at::kFloat, B, x));
  if (!THPVariable_Check(a[5])) set.min_p = share(a[5], "min_p", 1.0);
  at::Tensor tokens = optional(a[6], "tokens"), logprobs = optional(a[7], "logprobs");
  if (tokens.defined()) {
    setting(a[6], "tokens", at::kLong, B, x);
    apart(tokens, "tokens", x, "logits");
  }
  if (logprobs.defined()) {
    setting(a[7], "logprobs", at::kFloat, B, x);
    apart(logprobs, "logprobs", x, "logits");
    if (tokens.defined()) apart(logprobs, "logprobs", tokens, "tokens");
  }
  for (int i = 1; i < 6; ++i)
    if (THPVariable_Check(a[i])) {
      if (tokens.defined()) apart(tokens, "tokens", THPVariable_Unpack(a[i]), "a setting");
      if (logprobs.defined()) apart(logprobs, "logprobs", THPVariable_Unpack(a[i]), "a setting");
    }
  const c10::cuda::CUDAGuard guard(x.device());
  if (tokens.defined()) written(tokens);
  else tokens = at::empty({B}, x.options().dtype(at::kLong));
  if (logprobs.defined()) written(logprobs);
  else logprobs = at::empty({B}, x.options().dtype(at::kFloat));
  const lce_status_t st = lce_sample(ptr(x), ld, B, V, dt, static_cast<const float*>(u), &set,
                                     static_cast<int64_t*>(ptr(tokens)), static_cast<float*>(ptr(logprobs)),
                                     stream_of(x));
  return st == LCE_OK ? tuple_of(tokens, logprobs) : status(st);
}

template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGS, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name, args)                                                                     \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, args>)),    \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(linear_forward, 7), ENTRY(linear_backward, 8), ENTRY(gated_forward, 6),
                         ENTRY(gated_backward, 8), ENTRY(clip, 5), ENTRY(layer_norm_forward, 5),
                         ENTRY(layer_norm_backward, 8), ENTRY(embedding_forward, 6),
                         ENTRY(embedding_backward, 9), ENTRY(sample, 8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
