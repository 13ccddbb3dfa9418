// Python binding of the operators around the attention: argument checks,
// outputs from torch's allocator and the call of the C ABI (include/fbob.h) on
// the current stream of the tensors' device.  Their smallest calls last a few
// microseconds on the GPU, less than the same marshalling written in Python
// (layer norm of 8 rows: 15 us a call there).
//
// Module functions take positional arguments only and None for what is absent;
// the Python module in front of them has the signatures and the documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "fbob.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_check = nullptr;  // raises the package's error for a status

// A Python error has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* name, const char* what) {
  PyErr_Format(type, "%s: %s", name, what);
  throw Raised{};
}

const Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, name, "a tensor is needed");
  return &THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

int dtype_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::BFloat16) return FBOB_BF16;
  if (t.scalar_type() == ScalarType::Float) return FBOB_FP32;
  PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %s", name, c10::toString(t.scalar_type()));
  throw Raised{};
}

int device_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) raise(PyExc_ValueError, name, "all tensors must be on the same CUDA device");
  return t.get_device();
}

// One contiguous tensor argument (absent ones pass).
void check(const Tensor* t, const char* name, int device, ScalarType dtype, std::optional<at::IntArrayRef> shape) {
  if (!t) return;
  if (!t->is_cuda() || t->get_device() != device)
    raise(PyExc_ValueError, name, "all tensors must be on the same CUDA device");
  if (t->scalar_type() != dtype) {
    PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", name, c10::toString(dtype), c10::toString(t->scalar_type()));
    throw Raised{};
  }
  if (shape && t->sizes() != *shape) {
    PyErr_Format(PyExc_ValueError, "%s: expected shape %s, got %s", name, text(*shape).c_str(), text(t->sizes()).c_str());
    throw Raised{};
  }
  if (!t->is_contiguous()) raise(PyExc_ValueError, name, "must be contiguous");
}

Tensor fresh(const Tensor& like, at::IntArrayRef shape, ScalarType dtype) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
}

// The given output, checked, or a new one.
Tensor output(PyObject* given, const char* name, const Tensor& like, int device, at::IntArrayRef shape, ScalarType dtype) {
  if (given == Py_None) return fresh(like, shape, dtype);
  const Tensor* t = tensor(given, name);
  check(t, name, device, dtype, shape);
  return *t;
}

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* ptr(const std::optional<Tensor>& t) { return t ? t->data_ptr() : nullptr; }

PyObject* wrapped(const std::optional<Tensor>& t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}

template <typename... T>
PyObject* tuple_of(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(t));
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (PyObject* o : {wrapped(t)...}) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

void done(fbob_status s) {
  if (s == FBOB_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", (int)s);
  Py_XDECREF(r);
  if (r) raise(PyExc_RuntimeError, "fbob", fbob_last_error());
  throw Raised{};
}

// The device made current for a call, and its current stream.
struct Launch {
  std::optional<c10::cuda::CUDAGuard> guard;
  cudaStream_t stream;
  explicit Launch(int device) {
    if (c10::cuda::current_device() != device) guard.emplace((c10::DeviceIndex)device);
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  }
};

long long integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  (void)name;
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", want, n);
    throw Raised{};
  }
}

// --- rotary positions -----------------------------------------------------------------------------

void check_heads(const Tensor& t, const char* name, const Tensor& like, int device) {
  if (t.dim() != 4) raise(PyExc_ValueError, name, "must be [B, H, N, d]");
  if (!t.is_cuda() || t.get_device() != device)
    raise(PyExc_ValueError, name, "all tensors must be on the same CUDA device");
  if (t.scalar_type() != like.scalar_type()) {
    PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", name, c10::toString(like.scalar_type()),
                 c10::toString(t.scalar_type()));
    throw Raised{};
  }
  if (t.stride(3) != 1 && t.size(3) > 1) raise(PyExc_ValueError, name, "the columns of a head must be contiguous");
}

Tensor rotary_side(const Tensor& x, const char* name, PyObject* given, const char* out_name, const Tensor& like,
                   int device, fbob_rotary_heads* h) {
  check_heads(x, name, like, device);
  Tensor y;
  if (given == Py_None) {
    y = fresh(like, x.sizes(), like.scalar_type());
  } else {
    y = *tensor(given, out_name);
    check_heads(y, out_name, like, device);
    if (y.sizes() != x.sizes()) {
      PyErr_Format(PyExc_ValueError, "%s: expected shape %s, got %s", out_name, text(x.sizes()).c_str(),
                   text(y.sizes()).c_str());
      throw Raised{};
    }
  }
  if (x.size(1) > INT_MAX) raise(PyExc_ValueError, name, "sizes must fit 32 bits");
  h->x = x.data_ptr(), h->y = y.data_ptr(), h->H = (int)x.size(1);
  for (int i = 0; i < 3; ++i) h->x_stride[i] = x.stride(i), h->y_stride[i] = y.stride(i);
  return y;
}

// (description, Q, K, positions, offset, transpose, Qo, Ko)
PyObject* rotary_apply(PyObject* const* a, Py_ssize_t n) {
  count(n, 8);
  Py_buffer desc;
  if (PyObject_GetBuffer(a[0], &desc, PyBUF_SIMPLE) != 0) throw Raised{};
  struct Release {
    Py_buffer* b;
    ~Release() { PyBuffer_Release(b); }
  } release{&desc};
  if (desc.len != (Py_ssize_t)sizeof(fbob_rotary)) raise(PyExc_TypeError, "rotary", "a Rotary description is needed");
  const Tensor& Q = *tensor(a[1], "Q");
  const Tensor* K = tensor(a[2], "K", true);
  const Tensor* pos = tensor(a[3], "positions", true);
  if (Q.dim() != 4) raise(PyExc_ValueError, "Q", "must be [B, H, N, d]");
  const int dtype = dtype_code(Q, "Q"), device = device_of(Q, "Q");
  const int64_t B = Q.size(0), N = Q.size(2), d = Q.size(3);
  if (B > INT_MAX || N > INT_MAX || d > INT_MAX) raise(PyExc_ValueError, "Q", "sizes must fit 32 bits");
  fbob_rotary_heads h[2];
  Launch at(device);
  const std::optional<Tensor> Qo = rotary_side(Q, "Q", a[6], "Qo", Q, device, &h[0]);
  std::optional<Tensor> Ko;
  if (K) {
    if (K->dim() != 4 || K->size(0) != B || K->size(2) != N || K->size(3) != d) {
      PyErr_Format(PyExc_ValueError, "K: expected shape (%lld, Hk, %lld, %lld), got %s", (long long)B, (long long)N,
                   (long long)d, text(K->sizes()).c_str());
      throw Raised{};
    }
    Ko = rotary_side(*K, "K", a[7], "Ko", Q, device, &h[1]);
  } else if (a[7] != Py_None) {
    raise(PyExc_ValueError, "Ko", "given without K");
  }
  int size = 0;
  int64_t step = 0;
  if (pos) {
    if (pos->scalar_type() != ScalarType::Int && pos->scalar_type() != ScalarType::Long)
      raise(PyExc_TypeError, "positions", "must be int32 or int64");
    if (!pos->is_cuda() || pos->get_device() != device)
      raise(PyExc_ValueError, "positions", "all tensors must be on the same CUDA device");
    const bool each = pos->dim() == 2 && pos->size(0) == B && pos->size(1) == N;
    if (!each && !(pos->dim() == 1 && pos->size(0) == N)) {
      PyErr_Format(PyExc_ValueError, "positions: expected shape (%lld,) or (%lld, %lld), got %s", (long long)N,
                   (long long)B, (long long)N, text(pos->sizes()).c_str());
      throw Raised{};
    }
    if (pos->stride(pos->dim() - 1) != 1 && N > 1) raise(PyExc_ValueError, "positions", "must be contiguous");
    size = (int)pos->element_size();
    step = each && B > 1 ? pos->stride(0) : 0;
  }
  done(fbob_rotary_apply(static_cast<const fbob_rotary*>(desc.buf), (int)B, (int)N, (int)d, dtype, h, K ? 2 : 1, ptr(pos),
                         size, step, integer(a[4], "offset"), flag(a[5]), at.stream));
  return K ? tuple_of(Qo, Ko) : wrapped(Qo);
}

// --- layer norm -----------------------------------------------------------------------------------

ScalarType weight_type(const Tensor& x, std::initializer_list<const Tensor*> ws) {
  for (const Tensor* w : ws)
    if (w) return w->scalar_type();
  return x.scalar_type();
}

fbob_norm norm_for(const Tensor& x, ScalarType wt, double eps) {
  if (x.dim() < 1) raise(PyExc_ValueError, "x", "must have at least one dimension");
  fbob_norm p;
  const int64_t D = x.size(-1);
  if (D > INT_MAX) raise(PyExc_ValueError, "x", "sizes must fit 32 bits");
  p.rows = D ? x.numel() / D : 0;
  p.D = (int)D;
  p.dtype = dtype_code(x, "x");
  if (wt != ScalarType::BFloat16 && wt != ScalarType::Float) raise(PyExc_TypeError, "weight", "unsupported dtype");
  p.weight_dtype = wt == ScalarType::BFloat16 ? FBOB_BF16 : FBOB_FP32;
  p.eps = (float)eps;
  return p;
}

// The given workspace, checked, or a new one of `need` bytes.
std::optional<Tensor> workspace_of(PyObject* given, const Tensor& like, int device, size_t need, ScalarType dtype) {
  if (given != Py_None) {
    const Tensor* t = tensor(given, "workspace");
    check(t, "workspace", device, dtype, std::nullopt);
    return *t;
  }
  if (need == 0) return std::nullopt;
  const int64_t each = dtype == ScalarType::Float ? 4 : 1;
  return fresh(like, {(int64_t)(need + each - 1) / each}, dtype);
}
size_t bytes_of(const std::optional<Tensor>& t) { return t ? (size_t)t->numel() * t->element_size() : 0; }

// (x, weight, bias, eps, y, mean, rstd)
PyObject* layer_norm_fwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 7);
  const Tensor& x = *tensor(a[0], "x");
  const Tensor *w = tensor(a[1], "weight", true), *b = tensor(a[2], "bias", true);
  const ScalarType wt = weight_type(x, {w, b}), xt = x.scalar_type();
  const fbob_norm p = norm_for(x, wt, number(a[3]));
  const int device = device_of(x, "x");
  const at::IntArrayRef shape = x.sizes(), rows = shape.slice(0, shape.size() - 1), cols = shape.slice(shape.size() - 1);
  check(&x, "x", device, xt, std::nullopt);
  check(w, "weight", device, wt, cols);
  check(b, "bias", device, wt, cols);
  Launch at(device);
  const std::optional<Tensor> y = output(a[4], "y", x, device, shape, xt);
  const std::optional<Tensor> mean = output(a[5], "mean", x, device, rows, ScalarType::Float);
  const std::optional<Tensor> rstd = output(a[6], "rstd", x, device, rows, ScalarType::Float);
  done(fbob_layer_norm_fwd(&p, ptr(&x), ptr(w), ptr(b), ptr(y), (float*)ptr(mean), (float*)ptr(rstd), at.stream));
  return tuple_of(y, mean, rstd);
}

void check_norm(const Tensor& x, const Tensor* w, const Tensor& mean, const Tensor& rstd, const Tensor& dy, int device) {
  const at::IntArrayRef shape = x.sizes(), rows = shape.slice(0, shape.size() - 1), cols = shape.slice(shape.size() - 1);
  check(&x, "x", device, x.scalar_type(), std::nullopt);
  check(&mean, "mean", device, ScalarType::Float, rows);
  check(&rstd, "rstd", device, ScalarType::Float, rows);
  check(&dy, "dy", device, x.scalar_type(), shape);
  if (w) check(w, "weight", device, w->scalar_type(), cols);
}

// (x, weight, mean, rstd, dy, dx, dw, db, want dx, want dw, want db, bias type or None, workspace)
PyObject* layer_norm_bwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 13);
  const Tensor& x = *tensor(a[0], "x");
  const Tensor* w = tensor(a[1], "weight", true);
  const Tensor &mean = *tensor(a[2], "mean"), &rstd = *tensor(a[3], "rstd"), &dy = *tensor(a[4], "dy");
  const ScalarType xt = x.scalar_type();
  const ScalarType wt = w                ? w->scalar_type()
                        : a[11] == Py_None ? xt
                        : integer(a[11], "bias_dtype") == FBOB_BF16 ? ScalarType::BFloat16
                                                                    : ScalarType::Float;
  const fbob_norm p = norm_for(x, wt, 0.0);
  const int device = device_of(x, "x");
  check_norm(x, w, mean, rstd, dy, device);
  const at::IntArrayRef shape = x.sizes(), cols = shape.slice(shape.size() - 1);
  const bool want_dx = flag(a[8]), want_dw = flag(a[9]) && w, want_db = flag(a[10]);
  Launch at(device);
  std::optional<Tensor> dx, dw, db;
  if (want_dx) dx = output(a[5], "dx", x, device, shape, xt);
  if (want_dw) dw = output(a[6], "dw", x, device, cols, wt);
  if (want_db) db = output(a[7], "db", x, device, cols, wt);
  size_t need = 0;
  if (want_dw || want_db) need = fbob_layer_norm_workspace_bytes(&p) / (want_dw && want_db ? 1 : 2);
  const auto ws = workspace_of(a[12], x, device, need, ScalarType::Float);
  done(fbob_layer_norm_bwd(&p, ptr(&x), ptr(w), (const float*)ptr(&mean), (const float*)ptr(&rstd), ptr(&dy), ptr(dx),
                           ptr(dw), ptr(db), (float*)ptr(ws), bytes_of(ws), at.stream));
  return tuple_of(dx, dw, db);
}

// (x, weight, mean, rstd, dy, ux, uw, ub, gx, gw, gdy, want gx, want gw, want gdy, workspace)
PyObject* layer_norm_bob(PyObject* const* a, Py_ssize_t n) {
  count(n, 15);
  const Tensor& x = *tensor(a[0], "x");
  const Tensor* w = tensor(a[1], "weight", true);
  const Tensor &mean = *tensor(a[2], "mean"), &rstd = *tensor(a[3], "rstd"), &dy = *tensor(a[4], "dy");
  const Tensor& ux = *tensor(a[5], "ux");
  const Tensor *uw = tensor(a[6], "uw", true), *ub = tensor(a[7], "ub", true);
  const ScalarType xt = x.scalar_type(), wt = weight_type(x, {w, uw, ub});
  const fbob_norm p = norm_for(x, wt, 0.0);
  const int device = device_of(x, "x");
  check_norm(x, w, mean, rstd, dy, device);
  const at::IntArrayRef shape = x.sizes(), cols = shape.slice(shape.size() - 1);
  check(&ux, "ux", device, xt, shape);
  check(uw, "uw", device, wt, cols);
  check(ub, "ub", device, wt, cols);
  const bool want_gx = flag(a[11]), want_gw = flag(a[12]) && w, want_gdy = flag(a[13]);
  Launch at(device);
  std::optional<Tensor> gx, gw, gdy;
  if (want_gx) gx = output(a[8], "gx", x, device, shape, xt);
  if (want_gw) gw = output(a[9], "gw", x, device, cols, wt);
  if (want_gdy) gdy = output(a[10], "gdy", x, device, shape, xt);
  const auto ws = workspace_of(a[14], x, device, want_gw ? fbob_layer_norm_workspace_bytes(&p) / 2 : 0, ScalarType::Float);
  done(fbob_layer_norm_bob(&p, ptr(&x), ptr(w), (const float*)ptr(&mean), (const float*)ptr(&rstd), ptr(&dy), ptr(&ux),
                           ptr(uw), ptr(ub), ptr(gx), ptr(gw), ptr(gdy), (float*)ptr(ws), bytes_of(ws), at.stream));
  return tuple_of(gx, gw, gdy);
}

// --- cross entropy of a linear head -----------------------------------------------------------------

fbob_linear_ce ce_for(const Tensor& H, const Tensor& W, PyObject* ignore, long long piece) {
  if (H.dim() != 2 || W.dim() != 2 || H.size(1) != W.size(1)) {
    PyErr_Format(PyExc_ValueError, "H [T, D] and W [V, D] are needed, got %s and %s", text(H.sizes()).c_str(),
                 text(W.sizes()).c_str());
    throw Raised{};
  }
  if (H.size(0) > INT_MAX || H.size(1) > INT_MAX || W.size(0) > INT_MAX || piece > INT_MAX || piece < INT_MIN)
    raise(PyExc_ValueError, "H, W", "sizes must fit 32 bits");
  fbob_linear_ce p;
  p.T = (int)H.size(0), p.D = (int)H.size(1), p.V = (int)W.size(0);
  p.dtype = dtype_code(H, "H");
  p.ignore_index = integer(ignore, "ignore_index");
  p.piece = (int)piece;
  return p;
}

int check_ce(const Tensor& H, const Tensor& W, const Tensor& target, const Tensor* lse, const Tensor* g) {
  const int device = device_of(H, "H");
  const at::IntArrayRef rows = H.sizes().slice(0, 1);
  check(&H, "H", device, H.scalar_type(), std::nullopt);
  check(&W, "W", device, H.scalar_type(), std::nullopt);
  check(&target, "target", device, ScalarType::Long, rows);
  check(lse, "lse", device, ScalarType::Float, rows);
  check(g, "g", device, ScalarType::Float, rows);
  return device;
}

const long long* targets(const Tensor& t) { return static_cast<const long long*>(t.data_ptr()); }

// (H, W, target, ignore_index, loss, lse, workspace)
PyObject* linear_ce_fwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 7);
  const Tensor &H = *tensor(a[0], "H"), &W = *tensor(a[1], "W"), &y = *tensor(a[2], "target");
  const fbob_linear_ce p = ce_for(H, W, a[3], 0);
  const int device = check_ce(H, W, y, nullptr, nullptr);
  const at::IntArrayRef rows = H.sizes().slice(0, 1);
  Launch at(device);
  const std::optional<Tensor> loss = output(a[4], "loss", H, device, rows, ScalarType::Float);
  const std::optional<Tensor> lse = output(a[5], "lse", H, device, rows, ScalarType::Float);
  const auto ws = workspace_of(a[6], H, device, fbob_linear_ce_workspace_bytes(&p, 0), ScalarType::Byte);
  done(fbob_linear_ce_fwd(&p, ptr(&H), ptr(&W), targets(y), (float*)ptr(loss), (float*)ptr(lse), ptr(ws), bytes_of(ws),
                          at.stream));
  return tuple_of(loss, lse);
}

// (H, W, target, lse, g, ignore_index, piece, dH, dW, want dH, want dW, workspace)
PyObject* linear_ce_bwd(PyObject* const* a, Py_ssize_t n) {
  count(n, 12);
  const Tensor &H = *tensor(a[0], "H"), &W = *tensor(a[1], "W"), &y = *tensor(a[2], "target");
  const Tensor &lse = *tensor(a[3], "lse"), &g = *tensor(a[4], "g");
  const fbob_linear_ce p = ce_for(H, W, a[5], integer(a[6], "piece"));
  const int device = check_ce(H, W, y, &lse, &g);
  Launch at(device);
  std::optional<Tensor> dH, dW;
  if (flag(a[9])) dH = output(a[7], "dH", H, device, H.sizes(), H.scalar_type());
  if (flag(a[10])) dW = output(a[8], "dW", H, device, W.sizes(), H.scalar_type());
  const auto ws = workspace_of(a[11], H, device, fbob_linear_ce_workspace_bytes(&p, 1), ScalarType::Byte);
  done(fbob_linear_ce_bwd(&p, ptr(&H), ptr(&W), targets(y), (const float*)ptr(&lse), (const float*)ptr(&g), ptr(dH),
                          ptr(dW), ptr(ws), bytes_of(ws), at.stream));
  return tuple_of(dH, dW);
}

// (H, W, target, lse, g, UH, UW, ignore_index, piece, gH, gW, gg, want gH, want gW, want gg, workspace)
PyObject* linear_ce_bob(PyObject* const* a, Py_ssize_t n) {
  count(n, 16);
  const Tensor &H = *tensor(a[0], "H"), &W = *tensor(a[1], "W"), &y = *tensor(a[2], "target");
  const Tensor &lse = *tensor(a[3], "lse"), &g = *tensor(a[4], "g");
  const Tensor *UH = tensor(a[5], "UH", true), *UW = tensor(a[6], "UW", true);
  const fbob_linear_ce p = ce_for(H, W, a[7], integer(a[8], "piece"));
  const int device = check_ce(H, W, y, &lse, &g);
  check(UH, "UH", device, H.scalar_type(), H.sizes());
  check(UW, "UW", device, H.scalar_type(), W.sizes());
  Launch at(device);
  std::optional<Tensor> gH, gW, gg;
  if (flag(a[12])) gH = output(a[9], "gH", H, device, H.sizes(), H.scalar_type());
  if (flag(a[13])) gW = output(a[10], "gW", H, device, W.sizes(), H.scalar_type());
  if (flag(a[14])) gg = output(a[11], "gg", H, device, H.sizes().slice(0, 1), ScalarType::Float);
  const auto ws = workspace_of(a[15], H, device, fbob_linear_ce_workspace_bytes(&p, 2), ScalarType::Byte);
  done(fbob_linear_ce_bob(&p, ptr(&H), ptr(&W), targets(y), (const float*)ptr(&lse), (const float*)ptr(&g), ptr(UH),
                          ptr(UW), ptr(gH), ptr(gW), (float*)ptr(gg), ptr(ws), bytes_of(ws), at.stream));
  return tuple_of(gH, gW, gg);
}

// C++ and torch errors become Python's; none crosses into the interpreter.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_check, f);
  Py_RETURN_NONE;
}

#define ENTRY(f) {#f, (PyCFunction)(void (*)(void))entry<f>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    ENTRY(rotary_apply),   ENTRY(layer_norm_fwd), ENTRY(layer_norm_bwd), ENTRY(layer_norm_bob),
    ENTRY(linear_ce_fwd),  ENTRY(linear_ce_bwd),  ENTRY(linear_ce_bob),  {"set_check", set_check, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fbob_model", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fbob_model(void) { return PyModule_Create(&g_module); }
