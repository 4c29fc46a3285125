// vn_torch.cpp -- the centre network's calls on torch tensors, as a Python extension module.
//
// It checks and marshals arguments, allocates results and workspaces from torch's allocator
// and calls the C ABI of libvn.so on the tensors' current stream; it holds no arithmetic. The same
// work in Python over ctypes took 17.5 us of a GB300's host for a layer norm whose kernel
// takes 2.3 us, most of it in allocations and in ctypes.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>
#include <vector>

#include "vn.h"

namespace {

PyObject* g_error = nullptr;  // VNError of the package's ctypes module

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}

void check(vn_status status, const char* where) {
  if (status == VN_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(status), where)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

std::string text_of(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}
std::string text_of(at::ScalarType t) {
  return std::string("torch.") + (t == at::kFloat ? "float32" : t == at::kBFloat16 ? "bfloat16" : at::toString(t));
}
std::string text_of(const at::Device& d) { return d.str(); }

// A tensor on a CUDA device, made contiguous.
at::Tensor input(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (the library has no CPU path)");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (the library has no CPU path)");
  return t.is_contiguous() ? t : t.contiguous();
}
std::optional<at::Tensor> optional_input(PyObject* o, const char* name) {
  if (o == Py_None) return std::nullopt;
  return input(o, name);
}

vn_dtype dtype_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return VN_F32;
  if (t.scalar_type() == at::kBFloat16) return VN_BF16;
  raise(PyExc_TypeError, std::string(name) + ": dtype " + text_of(t.scalar_type()) + " is not supported (float32 or bfloat16)");
}

void beside(const at::Tensor& t, const at::Tensor& x) {
  if (t.device() != x.device())
    raise(PyExc_ValueError,
          "the tensors of one call must share a device, got " + text_of(x.device()) + " and " + text_of(t.device()));
}
void shaped(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape)
    raise(PyExc_ValueError, std::string(name) + " must have shape " + text_of(shape) + ", got " + text_of(t.sizes()));
}
// Of this shape, and of x's dtype and device.
void like(const at::Tensor& t, const char* name, at::IntArrayRef shape, const at::Tensor& x) {
  shaped(t, name, shape);
  if (t.scalar_type() != x.scalar_type())
    raise(PyExc_TypeError, std::string(name) + " must be " + text_of(x.scalar_type()) + ", got " + text_of(t.scalar_type()));
  beside(t, x);
}
// A parameter vector of n elements beside x.
void vector_of(const std::optional<at::Tensor>& t, const char* name, int64_t n, const at::Tensor& x) {
  if (!t) return;
  const int64_t want[1] = {n};
  shaped(*t, name, want);
  beside(*t, x);
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& x) {
  return at::detail::empty_cuda(shape, type, x.device(), std::nullopt);
}
// What a call writes over counts as changed in place, for autograd's check of what it has saved.
void changed(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
at::Tensor result(PyObject* out, at::IntArrayRef shape, const at::Tensor& x) {
  if (out == Py_None) return empty(shape, x.scalar_type(), x);
  if (THPVariable_Check(out)) {
    const at::Tensor& t = THPVariable_Unpack(out);
    if (t.sizes() == shape && t.scalar_type() == x.scalar_type() && t.is_contiguous() && t.device() == x.device()) {
      changed(t);
      return t;
    }
  }
  raise(PyExc_ValueError, "out must be a contiguous " + text_of(x.scalar_type()) + " tensor of shape " + text_of(shape) +
                              " on " + text_of(x.device()));
}
std::optional<at::Tensor> workspace(int64_t bytes, const at::Tensor& x) {
  if (bytes <= 0) return std::nullopt;
  const int64_t shape[1] = {bytes};
  return empty(shape, at::kByte, x);
}

void* at_(const at::Tensor& t) { return t.data_ptr(); }
void* at_(const std::optional<at::Tensor>& t) { return t ? t->data_ptr() : nullptr; }

// x's device made current, for as long as this lives, and its stream.
struct On {
  explicit On(const at::Tensor& x) {
    const c10::DeviceIndex want = x.device().index();
    was = c10::cuda::current_device();
    if (was != want) c10::cuda::set_device(want); else was = -1;
    stream = c10::cuda::getCurrentCUDAStream(want).stream();
  }
  ~On() {
    if (was >= 0) c10::cuda::set_device(was);
  }
  c10::DeviceIndex was;
  void* stream;
};

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}
int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (o == nullptr) throw Raised{};
  return o;
}
PyObject* wrap(const std::optional<at::Tensor>& t) {
  if (t) return wrap(*t);
  Py_RETURN_NONE;
}
template <typename... T>
PyObject* tuple(const T&... t) {
  PyObject* items[] = {wrap(t)...};
  PyObject* r = PyTuple_New(sizeof...(T));
  if (r == nullptr) throw Raised{};
  for (size_t i = 0; i < sizeof...(T); ++i) PyTuple_SET_ITEM(r, static_cast<Py_ssize_t>(i), items[i]);
  return r;
}

void counted(Py_ssize_t got, Py_ssize_t want, const char* name) {
  if (got != want) raise(PyExc_TypeError, std::string(name) + " takes " + std::to_string(want) + " arguments");
}

// The two tensors of a linear layer; rows, in, out, its type and the shape of its result.
struct Layer {
  Layer(PyObject* xo, PyObject* wo) : x(input(xo, "x")), w(input(wo, "weight")) {
    if (w.dim() != 2) raise(PyExc_ValueError, "weight must be (out_features, in_features)");
    n = w.size(0);
    k = w.size(1);
    if (x.dim() < 1 || x.size(-1) != k)
      raise(PyExc_ValueError, "x must be (..., " + std::to_string(k) + "), got " + text_of(x.sizes()));
    if (x.scalar_type() != w.scalar_type())
      raise(PyExc_TypeError, "x and weight must have one dtype, got " + text_of(x.scalar_type()) + " and " + text_of(w.scalar_type()));
    beside(w, x);
    dt = dtype_of(x, "x");
    rows = 1;
    for (int64_t i = 0; i + 1 < x.dim(); ++i) rows *= x.size(i);
    shape.assign(x.sizes().begin(), x.sizes().end());
    shape.back() = n;
  }
  at::Tensor x, w;
  int64_t rows, k, n;
  vn_dtype dt;
  c10::SmallVector<int64_t, 5> shape;
};

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// linear(x, weight, bias, activation, residual, preact, out) -> y or (y, z)
PyObject* linear(PyObject* const* a, Py_ssize_t count) {
  counted(count, 7, "linear");
  const Layer l(a[0], a[1]);
  const auto bias = optional_input(a[2], "bias");
  vector_of(bias, "bias", l.n, l.x);
  const auto residual = optional_input(a[4], "residual");
  if (residual) like(*residual, "residual", l.shape, l.x);
  const auto act = static_cast<vn_act>(whole(a[3]));
  const vn_dtype bias_dt = bias ? dtype_of(*bias, "bias") : VN_F32;
  const at::Tensor y = result(a[6], l.shape, l.x);
  std::optional<at::Tensor> z;
  if (truth(a[5])) z = empty(l.shape, l.x.scalar_type(), l.x);
  const int64_t need = vn_linear_workspace(l.rows, l.k, l.n, l.dt, aligned16(at_(l.x)) && aligned16(at_(l.w)));
  const auto ws = workspace(need, l.x);
  {
    const On on(l.x);
    check(vn_linear(at_(l.x), at_(l.w), l.dt, at_(bias), bias_dt, at_(residual), l.rows, l.k, l.n, act, at_(y), at_(z),
                    at_(ws), need > 0 ? need : 0, on.stream),
          "vn_linear");
  }
  return z ? tuple(y, z) : wrap(y);
}

// linear_backward(grad, x, weight, preact, activation, bias) -> (grad_x, grad_weight, grad_bias)
PyObject* linear_backward(PyObject* const* a, Py_ssize_t count) {
  counted(count, 6, "linear_backward");
  const Layer l(a[1], a[2]);
  const at::Tensor grad = input(a[0], "grad");
  like(grad, "grad", l.shape, l.x);
  const auto act = static_cast<vn_act>(whole(a[4]));
  std::optional<at::Tensor> z;
  if (act != VN_ACT_NONE) {
    if (a[3] == Py_None) raise(PyExc_ValueError, "the gradient through an activation needs preact");
    z = input(a[3], "preact");
    like(*z, "preact", l.shape, l.x);
  }
  const at::Tensor gx = empty(l.x.sizes(), l.x.scalar_type(), l.x), gw = empty(l.w.sizes(), l.x.scalar_type(), l.x);
  std::optional<at::Tensor> gb;
  const int64_t vector[1] = {l.n};
  if (truth(a[5])) gb = empty(vector, l.x.scalar_type(), l.x);
  const int64_t need = vn_linear_backward_workspace(
      l.rows, l.k, l.n, l.dt, act, aligned16(at_(grad)) && aligned16(at_(l.x)) && aligned16(at_(l.w)));
  const auto ws = workspace(need, l.x);
  {
    const On on(l.x);
    check(vn_linear_backward(at_(grad), at_(l.x), at_(l.w), at_(z), l.dt, l.rows, l.k, l.n, act, at_(gx), at_(gw),
                             at_(gb), l.dt, at_(ws), need > 0 ? need : 0, on.stream),
          "vn_linear_backward");
  }
  return tuple(gx, gw, gb);
}

// Rows and length of a norm's input.
int64_t norm_rows(const at::Tensor& x, int64_t* n) {
  if (x.dim() < 1 || x.size(-1) < 1) raise(PyExc_ValueError, "x must be (..., n) with n >= 1");
  *n = x.size(-1);
  int64_t rows = 1;
  for (int64_t i = 0; i + 1 < x.dim(); ++i) rows *= x.size(i);
  return rows;
}

// layer_norm(x, weight, bias, eps, out) -> (y, mean, rstd)
PyObject* layer_norm(PyObject* const* a, Py_ssize_t count) {
  counted(count, 5, "layer_norm");
  const at::Tensor x = input(a[0], "x");
  int64_t n;
  const int64_t rows = norm_rows(x, &n);
  const auto w = optional_input(a[1], "weight"), b = optional_input(a[2], "bias");
  vector_of(w, "weight", n, x);
  vector_of(b, "bias", n, x);
  const vn_dtype dt = dtype_of(x, "x");
  const vn_dtype wdt = w ? dtype_of(*w, "weight") : b ? dtype_of(*b, "bias") : VN_F32;
  if (w && b && w->scalar_type() != b->scalar_type()) raise(PyExc_TypeError, "weight and bias must have one dtype");
  const double eps = real(a[3]);
  const at::Tensor y = result(a[4], x.sizes(), x);
  const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
  const at::Tensor mean = empty(lead, at::kFloat, x), rstd = empty(lead, at::kFloat, x);
  {
    const On on(x);
    check(vn_layer_norm(at_(x), dt, at_(w), at_(b), wdt, rows, n, eps, at_(y), static_cast<float*>(at_(mean)),
                        static_cast<float*>(at_(rstd)), on.stream),
          "vn_layer_norm");
  }
  return tuple(y, mean, rstd);
}

// layer_norm_backward(grad, x, mean, rstd, weight) -> (grad_x, grad_weight, grad_bias)
PyObject* layer_norm_backward(PyObject* const* a, Py_ssize_t count) {
  counted(count, 5, "layer_norm_backward");
  const at::Tensor x = input(a[1], "x"), grad = input(a[0], "grad");
  int64_t n;
  const int64_t rows = norm_rows(x, &n);
  like(grad, "grad", x.sizes(), x);
  const at::Tensor mean = input(a[2], "mean"), rstd = input(a[3], "rstd");
  const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
  const at::Tensor* stats[2] = {&mean, &rstd};
  for (int i = 0; i < 2; ++i) {
    const char* name = i == 0 ? "mean" : "rstd";
    shaped(*stats[i], name, lead);
    if (stats[i]->scalar_type() != at::kFloat) raise(PyExc_TypeError, std::string(name) + " must be float32");
    beside(*stats[i], x);
  }
  const auto w = optional_input(a[4], "weight");
  vector_of(w, "weight", n, x);
  const vn_dtype dt = dtype_of(x, "x"), wdt = w ? dtype_of(*w, "weight") : VN_F32;
  const at::Tensor gx = empty(x.sizes(), x.scalar_type(), x);
  std::optional<at::Tensor> gw, gb, ws;
  int64_t need = 0;
  if (w) {
    gw = empty(w->sizes(), w->scalar_type(), x);
    gb = empty(w->sizes(), w->scalar_type(), x);
    need = vn_layer_norm_backward_workspace(rows, n);
    ws = workspace(need, x);
  }
  {
    const On on(x);
    check(vn_layer_norm_backward(at_(grad), at_(x), dt, static_cast<const float*>(at_(mean)),
                                 static_cast<const float*>(at_(rstd)), at_(w), wdt, rows, n, at_(gx), at_(gw), at_(gb),
                                 at_(ws), need > 0 ? need : 0, on.stream),
          "vn_layer_norm_backward");
  }
  return tuple(gx, gw, gb);
}

// adamw(params, grads, table, state_bits, lr, beta1, beta2, eps, step, maximize): one step of the
// tensors in the list `params`. grads: a list of as many, or one flat tensor. table: the
// address of a row of vn_adamw_tensor for each, in which only param and grad are set here.
PyObject* adamw(PyObject* const* a, Py_ssize_t count) {
  counted(count, 10, "adamw");
  PyObject* params = a[0];
  const Py_ssize_t n = PyList_GET_SIZE(params);
  auto* table = static_cast<vn_adamw_tensor*>(PyLong_AsVoidPtr(a[2]));
  if (table == nullptr) throw Raised{};
  const at::Tensor& first = THPVariable_Unpack(PyList_GET_ITEM(params, 0));
  std::vector<at::Tensor> kept;  // copies of gradients that were not contiguous
  at::ScalarType kind = at::kFloat;
  at::Tensor flat;
  char* at_flat = nullptr;
  const bool one = THPVariable_Check(a[1]);
  if (one) {
    flat = input(a[1], "grads");
    int64_t total = 0;
    for (Py_ssize_t i = 0; i < n; ++i) total += table[i].n;
    if (flat.dim() != 1 || flat.numel() != total)
      raise(PyExc_ValueError, "a flat gradient must have shape (" + std::to_string(total) + ",)");
    beside(flat, first);
    kind = flat.scalar_type();
    at_flat = static_cast<char*>(flat.data_ptr());
  } else {
    if (!PyList_Check(a[1])) raise(PyExc_TypeError, "grads must be a flat tensor or a sequence of tensors");
    if (PyList_GET_SIZE(a[1]) != n)
      raise(PyExc_ValueError, std::to_string(n) + " tensors but " + std::to_string(PyList_GET_SIZE(a[1])) + " gradients");
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor& p = THPVariable_Unpack(PyList_GET_ITEM(params, i));
    if (p.numel() != table[i].n || !p.is_contiguous() || p.scalar_type() != first.scalar_type() || p.device() != first.device())
      raise(PyExc_ValueError, "params[" + std::to_string(i) + "] is not the tensor that the handle was made for");
    table[i].param = p.data_ptr();
    if (one) {
      table[i].grad = at_flat;
      at_flat += table[i].n * flat.element_size();
      continue;
    }
    PyObject* o = PyList_GET_ITEM(a[1], i);
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).sizes() != p.sizes() || THPVariable_Unpack(o).device() != p.device())
      raise(PyExc_ValueError, "grads[" + std::to_string(i) + "] must have params[" + std::to_string(i) + "]'s shape and device");
    const at::Tensor& g = THPVariable_Unpack(o);
    if (i == 0) kind = g.scalar_type();
    else if (g.scalar_type() != kind) raise(PyExc_TypeError, "the gradients must have one dtype");
    if (g.is_contiguous()) {
      table[i].grad = g.data_ptr();
    } else {
      kept.push_back(g.contiguous());
      table[i].grad = kept.back().data_ptr();
    }
  }
  if (kind != at::kFloat && kind != at::kBFloat16)
    raise(PyExc_TypeError, "grads: dtype " + text_of(kind) + " is not supported (float32 or bfloat16)");
  const int bits = static_cast<int>(whole(a[3]));
  const double lr = real(a[4]), beta1 = real(a[5]), beta2 = real(a[6]), eps = real(a[7]);
  const int64_t step = whole(a[8]);
  const int maximize = truth(a[9]);
  {
    const On on(first);
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
      raise(PyExc_RuntimeError, "AdamW.step cannot be captured in a graph: its step number and learning rate would be "
                                "those of the capture in every replay");
    check(vn_adamw(table, n, dtype_of(first, "params"), kind == at::kBFloat16 ? VN_BF16 : VN_F32, bits, lr, beta1, beta2,
                   eps, step, maximize, on.stream),
          "vn_adamw");
  }
  for (Py_ssize_t i = 0; i < n; ++i) changed(THPVariable_Unpack(PyList_GET_ITEM(params, i)));
  Py_RETURN_NONE;
}

// adamw_moments(m, v, m_scale, v_scale) -> (m, v) in fp32
PyObject* adamw_moments(PyObject* const* a, Py_ssize_t count) {
  counted(count, 4, "adamw_moments");
  const at::Tensor m = input(a[0], "m"), v = input(a[1], "v"), ms = input(a[2], "m_scale"), vs = input(a[3], "v_scale");
  const at::Tensor mo = empty(m.sizes(), at::kFloat, m), vo = empty(m.sizes(), at::kFloat, m);
  {
    const On on(m);
    check(vn_adamw_moments(at_(m), at_(v), static_cast<const float*>(at_(ms)), static_cast<const float*>(at_(vs)),
                           m.numel(), static_cast<float*>(at_(mo)), static_cast<float*>(at_(vo)), on.stream),
          "vn_adamw_moments");
  }
  return tuple(mo, vo);
}

template <PyObject* (*kFn)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  try {
    return kFn(args, count);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*kFn)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFn>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<linear>("linear"),         method<linear_backward>("linear_backward"),
    method<layer_norm>("layer_norm"), method<layer_norm_backward>("layer_norm_backward"),
    method<adamw>("adamw"),           method<adamw_moments>("adamw_moments"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* lib = PyImport_ImportModule("virtual_noise_perturbed_gb300._lib");
  if (lib == nullptr) return nullptr;
  g_error = PyObject_GetAttrString(lib, "VNError");
  Py_DECREF(lib);
  return g_error == nullptr ? nullptr : PyModule_Create(&g_module);
}
