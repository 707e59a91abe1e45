// binding.cpp: the dense operators' arguments from Python to the C entry points
// (a CPython module linked against libmoe.so and torch).
//
// These calls take a few microseconds on the GPU, and checking a call's tensors in
// Python and passing them through ctypes took as long as that (a projection 8.2 us
// on the host, layer norm 6.4; 3.3 and 2.6 of them in the entry point).  What is
// checked and how it is refused is the same: ValueError for a tensor that is not
// as the call's sizes imply, the entry point's status for the rest.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/moe.h"

namespace {

using at::ScalarType;
using Shape = at::IntArrayRef;

struct Raised {};   // a Python error is set

[[noreturn]] void refuse(const std::string& what, PyObject* type = PyExc_ValueError) {
  PyErr_SetString(type, what.c_str());
  throw Raised();
}

std::string dtype_name(ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    default: return std::string("torch.") + c10::toString(t);
  }
}

std::string shape_name(Shape s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor* optional_tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name, PyExc_TypeError);
  return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = optional_tensor(o, name);
  if (!t) refuse(std::string(name) + " must be a tensor, got None", PyExc_TypeError);
  return *t;
}

// rows and columns of a matrix, as the entry points take them
struct Dims {
  int rows, cols;
  Dims(const at::Tensor& t, const char* name) {
    if (t.dim() != 2) refuse(std::string(name) + " must have 2 dimensions, got " + std::to_string(t.dim()));
    if (t.size(0) > INT_MAX || t.size(1) > INT_MAX) refuse(std::string(name) + " is too large: " + shape_name(t.sizes()));
    rows = (int)t.size(0);
    cols = (int)t.size(1);
  }
};

int dtype_code(const at::Tensor& t, const char* name, bool f32) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_BF16;
    case at::kHalf: return MOE_F16;
    case at::kFloat:
      if (f32) return MOE_F32;
      [[fallthrough]];
    default: break;
  }
  refuse(std::string(name) + " must be one of torch.bfloat16, torch.float16" + (f32 ? ", torch.float32" : "") + ", got " +
         dtype_name(t.scalar_type()));
}

struct Want {
  int64_t size[2];
  size_t dims;
  Want(int64_t n) : size{n, 0}, dims(1) {}
  Want(int64_t rows, int64_t cols) : size{rows, cols}, dims(2) {}
  Shape shape() const { return Shape(size, dims); }
};

struct Spec {
  const at::Tensor* t;   // null: not given
  const char* name;
  ScalarType dtype;
  Want want;
};

void check_one(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}

// Shapes first, then the rest; every tensor on the current device, which the kernel is launched on.
void check(std::initializer_list<Spec> specs, const at::Tensor* ws, const at::Tensor* status) {
  for (const Spec& s : specs)
    if (s.t && s.t->sizes() != s.want.shape())
      refuse(std::string(s.name) + " must have shape " + shape_name(s.want.shape()) + ", got " + shape_name(s.t->sizes()));
  if (status && status->numel() < 1) refuse("status must hold one int32");
  for (const Spec& s : specs)
    if (s.t) {
      check_one(*s.t, s.name);
      if (s.t->scalar_type() != s.dtype) refuse(std::string(s.name) + " must be " + dtype_name(s.dtype) + ", got " + dtype_name(s.t->scalar_type()));
    }
  if (status) {
    check_one(*status, "status");
    if (status->scalar_type() != at::kInt) refuse("status must be torch.int32, got " + dtype_name(status->scalar_type()));
  }
  if (ws) check_one(*ws, "ws");
  const int dev = c10::cuda::current_device();
  auto here = [&](const at::Tensor* t) {
    if (t && t->get_device() != dev)
      refuse("every tensor must be on the current device " + std::to_string(dev) + ", got one on " + t->device().str());
  };
  for (const Spec& s : specs) here(s.t);
  here(ws);
  here(status);
}

template <typename T = void>
T* ptr(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
template <typename T = void>
T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

moe_stream_t stream_of(PyObject* o) {
  if (o == Py_None) return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
  PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
  if (!s) throw Raised();
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw Raised();
  return reinterpret_cast<moe_stream_t>(p);
}

int to_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT_MIN || v > INT_MAX) refuse("integer out of range", PyExc_OverflowError);
  return (int)v;
}

// Runs `f` (arguments to status), with every C++ exception as a Python error.
template <typename F>
PyObject* entry(Py_ssize_t got, Py_ssize_t want, F&& f) {
  try {
    if (got != want) refuse("takes " + std::to_string(want) + " arguments, got " + std::to_string(got), PyExc_TypeError);
    return PyLong_FromLong(f());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The call itself, without the interpreter's lock.
template <typename F>
int unlocked(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  const int rc = f();
  PyEval_RestoreThread(s);
  return rc;
}

size_t bytes_of(const at::Tensor& t) { return (size_t)t.numel() * t.element_size(); }

// The type of the first of weight and bias (or their gradients) that is there; x's where none is.
ScalarType param_type(const at::Tensor& x, std::initializer_list<const at::Tensor*> params, const char* names) {
  for (const at::Tensor* p : params)
    if (p) {
      if (p->scalar_type() != x.scalar_type() && p->scalar_type() != at::kFloat)
        refuse(std::string(names) + " must be " + dtype_name(x.scalar_type()) + " or torch.float32, got " + dtype_name(p->scalar_type()));
      return p->scalar_type();
    }
  return x.scalar_type();
}

int param_code(ScalarType t) { return t == at::kBFloat16 ? MOE_BF16 : t == at::kHalf ? MOE_F16 : MOE_F32; }

// x, weight, bias, eps, y, mean, rstd, stream
PyObject* layernorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 8, [&] {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor *w = optional_tensor(a[1], "weight"), *b = optional_tensor(a[2], "bias"), *mean = optional_tensor(a[5], "mean"),
                     *rstd = optional_tensor(a[6], "rstd");
    const at::Tensor& y = tensor(a[4], "y");
    const Dims d(x, "x");
    const int dt = dtype_code(x, "x", true);
    const ScalarType t = x.scalar_type(), wt = param_type(x, {w, b}, "weight and bias");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    check({{&x, "x", t, {d.rows, d.cols}}, {w, "weight", wt, {d.cols}}, {b, "bias", wt, {d.cols}}, {&y, "y", t, {d.rows, d.cols}},
           {mean, "mean", at::kFloat, {d.rows}}, {rstd, "rstd", at::kFloat, {d.rows}}}, nullptr, nullptr);
    const moe_stream_t st = stream_of(a[7]);
    return unlocked([&] {
      return moe_layernorm(ptr(x), d.rows, d.cols, dt, ptr(w), ptr(b), param_code(wt), (float)eps, ptr(y), ptr<float>(mean), ptr<float>(rstd), st);
    });
  });
}

// dy, x, weight, mean, rstd, dx, dweight, dbias, ws, stream
PyObject* layernorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 10, [&] {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &mean = tensor(a[3], "mean"), &rstd = tensor(a[4], "rstd"),
                     &dx = tensor(a[5], "dx"), &ws = tensor(a[8], "ws");
    const at::Tensor *w = optional_tensor(a[2], "weight"), *dw = optional_tensor(a[6], "dweight"), *db = optional_tensor(a[7], "dbias");
    const Dims d(x, "x");
    const int dt = dtype_code(x, "x", true);
    const ScalarType t = x.scalar_type(), wt = param_type(x, {w, dw, db}, "weight, dweight and dbias");
    check({{&dy, "dy", t, {d.rows, d.cols}}, {&x, "x", t, {d.rows, d.cols}}, {w, "weight", wt, {d.cols}}, {&mean, "mean", at::kFloat, {d.rows}},
           {&rstd, "rstd", at::kFloat, {d.rows}}, {&dx, "dx", t, {d.rows, d.cols}}, {dw, "dweight", wt, {d.cols}}, {db, "dbias", wt, {d.cols}}},
          &ws, nullptr);
    const moe_stream_t st = stream_of(a[9]);
    return unlocked([&] {
      return moe_layernorm_bwd(ptr(dy), ptr(x), d.rows, d.cols, dt, ptr(w), param_code(wt), ptr<float>(mean), ptr<float>(rstd), ptr(dx), ptr(dw),
                               ptr(db), ptr(ws), bytes_of(ws), st);
    });
  });
}

// x, W, y, status, bias, residual, act, slope, stream
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 9, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &W = tensor(a[1], "W"), &y = tensor(a[2], "y"), &status = tensor(a[3], "status");
    const at::Tensor *b = optional_tensor(a[4], "bias"), *res = optional_tensor(a[5], "residual"), *slope = optional_tensor(a[7], "slope");
    const int act = to_int(a[6]);
    const Dims d(x, "x");
    const int N = Dims(W, "W").rows, dt = dtype_code(x, "x", false);
    const ScalarType t = x.scalar_type();
    check({{&x, "x", t, {d.rows, d.cols}}, {&W, "W", t, {N, d.cols}}, {&y, "y", t, {d.rows, N}}, {b, "bias", t, {N}},
           {res, "residual", t, {d.rows, N}}, {slope, "slope", t, {d.rows, N}}}, nullptr, &status);
    const moe_stream_t st = stream_of(a[8]);
    return unlocked([&] {
      return moe_linear(ptr(x), d.rows, d.cols, ptr(W), N, dt, ptr(b), ptr(res), act, ptr(y), ptr(slope), ptr<int32_t>(status), st);
    });
  });
}

// dy, x, W, dx, dW, ws, status, dbias, slope, stream
PyObject* linear_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 10, [&] {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &W = tensor(a[2], "W"), &ws = tensor(a[5], "ws"), &status = tensor(a[6], "status");
    const at::Tensor *dx = optional_tensor(a[3], "dx"), *dW = optional_tensor(a[4], "dW"), *db = optional_tensor(a[7], "dbias"),
                     *slope = optional_tensor(a[8], "slope");
    const Dims d(x, "x");
    const int N = Dims(W, "W").rows, dt = dtype_code(x, "x", false);
    const ScalarType t = x.scalar_type();
    check({{&dy, "dy", t, {d.rows, N}}, {&x, "x", t, {d.rows, d.cols}}, {&W, "W", t, {N, d.cols}}, {dx, "dx", t, {d.rows, d.cols}},
           {dW, "dW", t, {N, d.cols}}, {db, "dbias", t, {N}}, {slope, "slope", t, {d.rows, N}}}, &ws, &status);
    const moe_stream_t st = stream_of(a[9]);
    return unlocked([&] {
      return moe_linear_bwd(ptr(dy), ptr(x), d.rows, d.cols, ptr(W), N, dt, ptr(slope), ptr(dx), ptr(dW), ptr(db), ptr(ws), bytes_of(ws),
                            ptr<int32_t>(status), st);
    });
  });
}

// x, W1, h, status, act, factors, stream
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &W1 = tensor(a[1], "W1"), &h = tensor(a[2], "h"), &status = tensor(a[3], "status");
    const at::Tensor* factors = optional_tensor(a[5], "factors");
    const int act = to_int(a[4]);
    const Dims d(x, "x");
    const int F = Dims(h, "h").cols, dt = dtype_code(x, "x", false);
    const ScalarType t = x.scalar_type();
    check({{&x, "x", t, {d.rows, d.cols}}, {&W1, "W1", t, {2LL * F, d.cols}}, {&h, "h", t, {d.rows, F}}, {factors, "factors", t, {d.rows, 2LL * F}}},
          nullptr, &status);
    const moe_stream_t st = stream_of(a[6]);
    return unlocked([&] { return moe_gated(ptr(x), d.rows, d.cols, ptr(W1), F, dt, act, ptr(h), ptr(factors), ptr<int32_t>(status), st); });
  });
}

// dh, x, W1, factors, dx, dW1, ws, status, stream
PyObject* gated_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 9, [&] {
    const at::Tensor &dh = tensor(a[0], "dh"), &x = tensor(a[1], "x"), &W1 = tensor(a[2], "W1"), &factors = tensor(a[3], "factors"),
                     &ws = tensor(a[6], "ws"), &status = tensor(a[7], "status");
    const at::Tensor *dx = optional_tensor(a[4], "dx"), *dW1 = optional_tensor(a[5], "dW1");
    const Dims d(x, "x");
    const int F = Dims(dh, "dh").cols, dt = dtype_code(x, "x", false);
    const ScalarType t = x.scalar_type();
    check({{&dh, "dh", t, {d.rows, F}}, {&x, "x", t, {d.rows, d.cols}}, {&W1, "W1", t, {2LL * F, d.cols}}, {&factors, "factors", t, {d.rows, 2LL * F}},
           {dx, "dx", t, {d.rows, d.cols}}, {dW1, "dW1", t, {2LL * F, d.cols}}}, &ws, &status);
    const moe_stream_t st = stream_of(a[8]);
    return unlocked([&] {
      return moe_gated_bwd(ptr(dh), ptr(x), d.rows, d.cols, ptr(W1), F, dt, ptr(factors), ptr(dx), ptr(dW1), ptr(ws), bytes_of(ws),
                           ptr<int32_t>(status), st);
    });
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<layernorm>("layernorm"), method<layernorm_bwd>("layernorm_bwd"), method<linear>("linear"),
                         method<linear_bwd>("linear_bwd"), method<gated>("gated"), method<gated_bwd>("gated_bwd"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
