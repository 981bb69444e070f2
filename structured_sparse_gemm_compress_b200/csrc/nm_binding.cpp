// nm_binding.cpp -- the Python binding of the calls whose own host time is a large
// part of a small problem: the feed-forward block and the microscaled products.
// It does what the ctypes binding does for the other calls -- check the tensors,
// allocate what is not given, pass pointers and the stream to the C ABI -- in a
// quarter of the time (quantisation of a few rows: 9 us a call through ctypes and
// torch.empty, of which the launch is 3).  No arithmetic happens here.
//
// The library is not linked: init() takes the addresses of its functions, so the
// module and ctypes always speak to the same copy.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "nmspmm.h"

namespace {

struct Api {
  decltype(&nm_mx_quantize) mx_quantize;
  decltype(&nm_mx_dequantize) mx_dequantize;
  decltype(&nm_spmm_mx) spmm_mx;
  decltype(&nm_spmm_mx_gated) spmm_mx_gated;
  decltype(&nm_spmm_gated) spmm_gated;
  decltype(&nm_gated_backward) gated_backward;
  decltype(&nm_gated_backward_workspace) gated_backward_workspace;
} api;

PyObject* g_raise = nullptr;  // raises NMError for a status

struct Refused {  // becomes a ValueError
  std::string what;
};
struct PythonError {};  // the Python error is set already

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

// A contiguous tensor of this type and shape on the current CUDA device.
void check(const at::Tensor& t, const char* name, at::ScalarType dt, at::IntArrayRef shape) {
  if (t.scalar_type() != dt || t.sizes() != shape || !t.is_contiguous())
    throw Refused{std::string(name) + " must be a contiguous " + shape_text(shape) + " tensor of type " + c10::toString(dt)};
  if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
    throw Refused{std::string(name) + " must be on the current CUDA device"};
}

// The stream of a call: None (the current one), a torch.cuda.Stream, or a raw handle.
// While it lives, outputs are allocated for that stream, so torch's allocator never
// hands their memory to work that is not ordered behind it.
struct CallStream {
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  cudaStream_t raw = nullptr;
  explicit CallStream(PyObject* o) {
    const auto dev = c10::cuda::current_device();
    if (o == Py_None) {
      raw = c10::cuda::getCurrentCUDAStream(dev).stream();
      return;
    }
    PyObject* v = o;
    if (!PyLong_Check(o)) {
      v = PyObject_GetAttrString(o, "cuda_stream");
      if (!v) throw PythonError{};
    } else {
      Py_INCREF(v);
    }
    raw = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
    Py_DECREF(v);
    if (PyErr_Occurred()) throw PythonError{};
    guard.emplace(raw ? c10::cuda::getStreamFromExternal(raw, dev) : c10::cuda::getDefaultCUDAStream(dev));
  }
};

at::Tensor make(at::IntArrayRef shape, at::ScalarType dt) {
  return at::detail::empty_cuda(shape, dt, c10::Device(c10::kCUDA, c10::cuda::current_device()), std::nullopt);
}

// The given tensor after checking it, or a new one.
at::Tensor given_or_new(PyObject* o, const char* name, at::ScalarType dt, at::IntArrayRef shape) {
  if (o == Py_None) return make(shape, dt);
  const at::Tensor& t = tensor(o, name);
  check(t, name, dt, shape);
  return t;
}

const float* vector(PyObject* o, const char* name, int64_t n) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  check(t, name, at::kFloat, {n});
  return t.const_data_ptr<float>();
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
void* pointer(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw PythonError{};
  return p;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return (float)v;
}

void status(nm_status st) {
  if (st == NM_OK) return;
  PyObject* r = PyObject_CallFunction(g_raise, "i", (int)st);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "a library call failed");
  throw PythonError{};
}

at::ScalarType scalar_type(int code) {
  switch (code) {
    case NM_INT8: return at::kChar;
    case NM_FP16: return at::kHalf;
    case NM_BF16: return at::kBFloat16;
    default: return at::kFloat;
  }
}

int float_code(at::ScalarType t, const char* what) {
  switch (t) {
    case at::kHalf: return NM_FP16;
    case at::kBFloat16: return NM_BF16;
    case at::kFloat: return NM_FP32;
    default: throw Refused{what};
  }
}

// Element type of an output: code of nm_out_type, `dflt` for the default.
at::ScalarType out_type(int64_t out, at::ScalarType dflt) {
  switch (out) {
    case NM_OUT_INT32: return at::kInt;
    case NM_OUT_FP32: return at::kFloat;
    case NM_OUT_FP16: return at::kHalf;
    case NM_OUT_BF16: return at::kBFloat16;
    case NM_OUT_INT8: return at::kChar;
    default: return dflt;
  }
}

int64_t scale_bytes(int64_t rows, int64_t k) { return (rows + 127) / 128 * ((k + 255) / 256) * 1024; }

struct Quantised {
  int64_t T, k;
  const void *q, *s;
};
Quantised quantised(PyObject* qo, PyObject* so) {
  const at::Tensor &Q = tensor(qo, "Q"), &S = tensor(so, "S");
  if (Q.dim() != 2) throw Refused{"Q must be [T, k / 2]"};
  const int64_t T = Q.size(0), half = Q.size(1);
  check(Q, "Q", at::kByte, {T, half});
  check(S, "S", at::kByte, {scale_bytes(T, 2 * half)});
  return {T, 2 * half, Q.const_data_ptr(), S.const_data_ptr()};
}

// The interpreter is free while the library launches (a full launch queue blocks).
template <typename F>
nm_status released(F f) {
  PyThreadState* t = PyEval_SaveThread();
  const nm_status st = f();
  PyEval_RestoreThread(t);
  return st;
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const PythonError&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* wrap(at::Tensor t, PyObject* given) {  // a given tensor is returned as the object it came in
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(std::move(t));
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
  return false;
}

// (X, Q, S, stream) -> (Q, S)
PyObject* mx_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  return guarded([&]() -> PyObject* {
    static const char* kWhat = "X must be a [T, k] float32/float16/bfloat16 tensor with contiguous rows";
    const at::Tensor& X = tensor(a[0], "X");
    const int dt = float_code(X.scalar_type(), kWhat);
    if (X.dim() != 2) throw Refused{kWhat};
    const int64_t T = X.size(0), k = X.size(1);
    if (k > 1 && X.stride(1) != 1) throw Refused{kWhat};
    if (!X.is_cuda() || X.get_device() != c10::cuda::current_device())
      throw Refused{"X must be on the current CUDA device"};
    CallStream s(a[3]);
    at::Tensor Q = given_or_new(a[1], "Q", at::kByte, {T, k / 2});
    at::Tensor S = given_or_new(a[2], "S", at::kByte, {scale_bytes(T, k)});
    status(released([&] {
      return api.mx_quantize(X.const_data_ptr(), T, k, T > 1 ? X.stride(0) : k, (nm_dtype)dt, Q.data_ptr(), S.data_ptr(),
                             s.raw);
    }));
    PyObject* t = PyTuple_New(2);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, wrap(std::move(Q), a[1]));
    PyTuple_SET_ITEM(t, 1, wrap(std::move(S), a[2]));
    return t;
  });
}

// (Q, S, dtype code, X, stream) -> X
PyObject* mx_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Quantised q = quantised(a[0], a[1]);
    const int dt = (int)integer(a[2]);
    CallStream s(a[4]);
    at::Tensor X = given_or_new(a[3], "X", scalar_type(dt), {q.T, q.k});
    status(released([&] { return api.mx_dequantize(q.q, q.s, q.T, q.k, (nm_dtype)dt, X.data_ptr(), s.raw); }));
    return wrap(std::move(X), a[3]);
  });
}

// (handle, n_out, k, source dtype code, gated, Q, S, Y, scale, bias, act, out, stream) -> Y
PyObject* spmm_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const nm_handle* h = static_cast<const nm_handle*>(pointer(a[0]));
    const int64_t n_out = integer(a[1]), k = integer(a[2]), src = integer(a[3]), gated = integer(a[4]);
    const Quantised q = quantised(a[5], a[6]);
    if (q.k != k) throw Refused{"Q holds k = " + std::to_string(q.k) + ", the handle " + std::to_string(k)};
    nm_epilogue ep{};
    ep.scale = vector(a[8], "scale", n_out);
    ep.bias = vector(a[9], "bias", n_out);
    ep.act = (nm_act)integer(a[10]);
    ep.out = (nm_out_type)integer(a[11]);
    ep.out_scale = 1.0f;
    CallStream s(a[12]);
    at::Tensor Y = given_or_new(a[7], "Y", out_type(ep.out, scalar_type((int)src)), {q.T, gated ? n_out / 2 : n_out});
    auto product = gated ? api.spmm_mx_gated : api.spmm_mx;
    status(released([&] { return product(h, q.q, q.s, q.T, Y.data_ptr(), &ep, s.raw); }));
    return wrap(std::move(Y), a[7]);
  });
}

// (handle, n_out, k, dtype code, X, Y, P, scale, bias, act, out, out_scale, stream) -> Y
PyObject* spmm_gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const nm_handle* h = static_cast<const nm_handle*>(pointer(a[0]));
    const int64_t n_out = integer(a[1]), k = integer(a[2]);
    const at::ScalarType dt = scalar_type((int)integer(a[3]));
    const at::Tensor& X = tensor(a[4], "X");
    if (X.dim() != 2) throw Refused{"X must be [T, k]"};
    const int64_t T = X.size(0);
    check(X, "X", dt, {T, k});
    nm_epilogue ep{};
    ep.scale = vector(a[7], "scale", n_out);
    ep.bias = vector(a[8], "bias", n_out);
    ep.act = (nm_act)integer(a[9]);
    ep.out = (nm_out_type)integer(a[10]);
    ep.out_scale = number(a[11]);
    void* P = nullptr;
    if (a[6] != Py_None) {
      const at::Tensor& p = tensor(a[6], "P");
      check(p, "P", dt, {T, n_out});
      P = p.data_ptr();
    }
    CallStream s(a[12]);
    at::Tensor Y = given_or_new(a[5], "Y", out_type(ep.out, dt == at::kChar ? at::kFloat : dt), {T, n_out / 2});
    status(released([&] { return api.spmm_gated(h, X.const_data_ptr(), T, Y.data_ptr(), P, &ep, s.raw); }));
    return wrap(std::move(Y), a[5]);
  });
}

// (handle, n_out, k, dtype code, X, P, dY, act, bias_grad, dX, dW, dbias, workspace, stream) -> (dX, dW, dbias)
PyObject* gated_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 14)) return nullptr;
  return guarded([&]() -> PyObject* {
    const nm_handle* h = static_cast<const nm_handle*>(pointer(a[0]));
    const int64_t n_out = integer(a[1]), k = integer(a[2]);
    const at::ScalarType dt = scalar_type((int)integer(a[3]));
    const at::Tensor &X = tensor(a[4], "X"), &P = tensor(a[5], "P"), &dY = tensor(a[6], "dY");
    if (X.dim() != 2) throw Refused{"X must be [T, k]"};
    const int64_t T = X.size(0);
    check(X, "X", dt, {T, k});
    check(P, "P", dt, {T, n_out});
    check(dY, "dY", dt, {T, n_out / 2});
    const int64_t act = integer(a[7]);
    const bool want_bias = integer(a[8]) != 0 || a[11] != Py_None;
    CallStream s(a[13]);
    at::Tensor dX = given_or_new(a[9], "dX", dt, {T, k}), dW = given_or_new(a[10], "dW", dt, {n_out, k}), dbias;
    if (want_bias) dbias = given_or_new(a[11], "dbias", at::kFloat, {n_out});
    at::Tensor ws;
    if (a[12] != Py_None) {
      ws = tensor(a[12], "workspace");
      check(ws, "workspace", at::kByte, {ws.numel()});
    } else {
      size_t bytes = 0;
      status(api.gated_backward_workspace(h, T, &bytes));
      ws = make({(int64_t)bytes}, at::kByte);
    }
    status(released([&] {
      return api.gated_backward(h, X.const_data_ptr(), P.const_data_ptr(), dY.const_data_ptr(), T, (nm_act)act,
                                dX.data_ptr(), dW.data_ptr(),
                                want_bias ? static_cast<float*>(dbias.data_ptr()) : nullptr, ws.data_ptr(),
                                (size_t)ws.numel(), s.raw);
    }));
    PyObject* t = PyTuple_New(3);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, wrap(std::move(dX), a[9]));
    PyTuple_SET_ITEM(t, 1, wrap(std::move(dW), a[10]));
    if (want_bias) {
      PyTuple_SET_ITEM(t, 2, wrap(std::move(dbias), a[11]));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(t, 2, Py_None);
    }
    return t;
  });
}

// init(raise, addresses): the function that raises for a status, and the library's
// functions in the order of Api.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    Py_INCREF(a[0]);
    Py_XSETREF(g_raise, a[0]);
    api.mx_quantize = reinterpret_cast<decltype(api.mx_quantize)>(pointer(a[1]));
    api.mx_dequantize = reinterpret_cast<decltype(api.mx_dequantize)>(pointer(a[2]));
    api.spmm_mx = reinterpret_cast<decltype(api.spmm_mx)>(pointer(a[3]));
    api.spmm_mx_gated = reinterpret_cast<decltype(api.spmm_mx_gated)>(pointer(a[4]));
    api.spmm_gated = reinterpret_cast<decltype(api.spmm_gated)>(pointer(a[5]));
    api.gated_backward = reinterpret_cast<decltype(api.gated_backward)>(pointer(a[6]));
    api.gated_backward_workspace = reinterpret_cast<decltype(api.gated_backward_workspace)>(pointer(a[7]));
    Py_RETURN_NONE;
  });
}

#define NM_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {NM_METHOD(init),       NM_METHOD(mx_quantize), NM_METHOD(mx_dequantize), NM_METHOD(spmm_mx),
                         NM_METHOD(spmm_gated), NM_METHOD(gated_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
