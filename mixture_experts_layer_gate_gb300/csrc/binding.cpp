// Python entries of the operators around the layer: argument checks on torch
// tensors, then the C call.  In Python the checks of seven tensors and the call
// through ctypes took 5.4 us of a launch's 7.5 (add_rms_norm, one row); here 0.4.
// Python keeps the names, defaults and documentation (binding.py).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/moe.h"

namespace {

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const std::string& text) {
  PyErr_SetString(PyExc_ValueError, text.c_str());
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: a torch tensor", what);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

// What the elements have to be.
struct Type {
  at::ScalarType first, second;
  Type(at::ScalarType t) : first(t), second(t) {}
  Type(at::ScalarType t, at::ScalarType u) : first(t), second(u) {}
};
const Type kFloat(at::ScalarType::Float), kBf16(at::ScalarType::BFloat16);
const Type kCodes(at::ScalarType::Byte, at::ScalarType::Float8_e4m3fn);

// of a moe_dtype_t; one that is none is left to the C call, which refuses it
Type type_of(int dtype) {
  switch (dtype) {
    case MOE_T_BF16: return kBf16;
    case MOE_T_F16: return at::ScalarType::Half;
    case MOE_T_F32: return kFloat;
    default: return at::ScalarType::Undefined;
  }
}

std::string name_of(const Type& type) {
  const std::string s = at::toString(type.first);
  return type.first == type.second ? s : s + " or " + at::toString(type.second);
}
bool is_of(const at::Tensor& t, const Type& type) {
  const at::ScalarType s = t.scalar_type();
  return s == type.first || s == type.second || type.first == at::ScalarType::Undefined;
}
// The kernels are launched on the current device, which a call looks up once (for
// each of seven tensors: 0.3 us).
thread_local int device_of_call = -1;
int current_device() {
  if (device_of_call < 0) device_of_call = c10::cuda::current_device();
  return device_of_call;
}
bool is_here(const at::Tensor& t) { return t.is_cuda() && t.get_device() == current_device(); }

struct Rows {
  void* p = nullptr;
  int64_t stride = 0;
  float* f32() const { return static_cast<float*>(p); }
};

// [rows, cols]; None stays null
Rows rows(PyObject* o, int64_t n, int64_t cols, const Type& type, const char* what) {
  Rows r;
  if (o == Py_None) return r;
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != cols || !is_of(t, type) || !is_here(t))
    refuse(std::string(what) + ": a tensor [" + std::to_string(n) + ", " + std::to_string(cols) + "] of " +
           name_of(type) + " on the current CUDA device");
  if (t.stride(1) != 1 && cols > 1) refuse(std::string(what) + ": adjacent columns");
  r.p = t.data_ptr();
  r.stride = n > 1 ? t.stride(0) : cols;
  return r;
}

// a contiguous tensor of n elements; None stays null
void* flat(PyObject* o, int64_t n, const Type& type, const char* what) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, what);
  if (t.numel() != n || !is_of(t, type) || !is_here(t) || !t.is_contiguous())
    refuse(std::string(what) + ": a contiguous tensor of " + std::to_string(n) + " elements of " + name_of(type) +
           " on the current CUDA device");
  return t.data_ptr();
}

struct Workspace {
  void* p;
  size_t bytes;
  explicit Workspace(PyObject* o) {
    const at::Tensor& t = tensor(o, "ws");
    if (!is_here(t) || !t.is_contiguous()) refuse("ws: a contiguous tensor on the current CUDA device");
    p = t.data_ptr();
    bytes = t.nbytes();
  }
};

// A copy of a ctypes structure: the problem, or pointers to weights.
template <typename T>
T problem(PyObject* o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Refused();
  const bool fits = b.len == static_cast<Py_ssize_t>(sizeof(T));
  T v{};
  if (fits) v = *static_cast<const T*>(b.buf);
  PyBuffer_Release(&b);
  if (!fits) refuse("not the structure of this call");
  return v;
}

// the given raw stream, or the current one of the current device
moe_stream_t stream_of(PyObject* o) {
  if (o == Py_None) return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(current_device()).stream());
  PyObject* i = PyNumber_Long(o);
  if (i == nullptr) throw Refused();
  const unsigned long long v = PyLong_AsUnsignedLongLong(i);
  Py_DECREF(i);
  if (PyErr_Occurred()) throw Refused();
  return reinterpret_cast<moe_stream_t>(v);
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// Runs f(arguments, ...) -> moe_status_t; C++ exceptions become Python's.
template <typename Fn>
PyObject* run(Py_ssize_t given, Py_ssize_t wanted, Fn&& f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments", wanted);
    return nullptr;
  }
  device_of_call = -1;
  try {
    return PyLong_FromLong(f());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The C call without the interpreter's lock: a full launch queue makes it wait.
template <typename Fn>
moe_status_t unlocked(Fn&& f) {
  moe_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return st;
}

// problem, x, weight, residual, residual_out, y, codes, scales, stream
PyObject* add_rms_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run(n, 9, [&] {
    const moe_norm_t p = problem<moe_norm_t>(v[0]);
    const int64_t T = p.T, H = p.H;
    const Type b = type_of(p.dtype);
    const Rows x = rows(v[1], T, H, b, "x"), r = rows(v[3], T, H, b, "residual");
    const Rows o = rows(v[4], T, H, b, "residual_out"), y = rows(v[5], T, H, b, "y");
    void* w = flat(v[2], H, type_of(p.weight_dtype), "weight");
    void* codes = flat(v[6], T * H, kCodes, "codes");
    void* scales = flat(v[7], T * (p.quant == MOE_QUANT_BLOCK128 ? blocks(H) : 1), kFloat, "scales");
    const moe_stream_t s = stream_of(v[8]);
    return unlocked([&] {
      return moe_add_rms_norm(&p, x.p, x.stride, r.p, r.stride, w, o.p, o.stride, y.p, y.stride, codes,
                              static_cast<float*>(scales), s);
    });
  });
}

// problem, x, w, logits, ws, stream
PyObject* router_logits(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run(n, 6, [&] {
    const moe_router_t p = problem<moe_router_t>(v[0]);
    const Type b = type_of(p.dtype);
    const Rows x = rows(v[1], p.T, p.H, b, "x"), w = rows(v[2], p.E, p.H, b, "w");
    void* logits = flat(v[3], static_cast<int64_t>(p.T) * p.E, kFloat, "logits");
    const Workspace ws(v[4]);
    const moe_stream_t s = stream_of(v[5]);
    return unlocked([&] {
      return moe_router_logits(&p, x.p, x.stride, w.p, w.stride, static_cast<float*>(logits), ws.p, ws.bytes, s);
    });
  });
}

// problem, a, a_scale, w, w_scale, out, ws, stream
PyObject* gemm_fp8_block(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run(n, 8, [&] {
    const moe_fp8_gemm_t p = problem<moe_fp8_gemm_t>(v[0]);
    const int64_t kb = blocks(p.K);
    const Rows a = rows(v[1], p.M, p.K, kCodes, "a"), as = rows(v[2], p.M, kb, kFloat, "a_scale");
    const Rows w = rows(v[3], p.N, p.K, kCodes, "w"), o = rows(v[5], p.M, p.N, type_of(p.out_dtype), "out");
    void* sw = flat(v[4], blocks(p.N) * kb, kFloat, "w_scale");
    const Workspace ws(v[6]);
    const moe_stream_t s = stream_of(v[7]);
    return unlocked([&] {
      return moe_gemm_fp8_block(&p, a.p, a.stride, as.f32(), as.stride, w.p, w.stride, static_cast<float*>(sw), o.p,
                                o.stride, ws.p, ws.bytes, s);
    });
  });
}

// problem, a, a_scale, w13, w13_scale, codes, scales, ws, stream
PyObject* gemm_fp8_block_swiglu(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run(n, 9, [&] {
    const moe_fp8_gemm_t p = problem<moe_fp8_gemm_t>(v[0]);
    const int64_t kb = blocks(p.K), N = p.N;
    const Rows a = rows(v[1], p.M, p.K, kCodes, "a"), as = rows(v[2], p.M, kb, kFloat, "a_scale");
    const Rows w = rows(v[3], 2 * N, p.K, kCodes, "w13");
    void* sw = flat(v[4], blocks(2 * N) * kb, kFloat, "w13_scale");
    void* codes = flat(v[5], p.M * N, kCodes, "codes");
    void* scales = flat(v[6], p.M * (N / 128), kFloat, "scales");
    const Workspace ws(v[7]);
    const moe_stream_t s = stream_of(v[8]);
    return unlocked([&] {
      return moe_gemm_fp8_block_swiglu(&p, a.p, a.stride, as.f32(), as.stride, w.p, w.stride, static_cast<float*>(sw),
                                       codes, static_cast<float*>(scales), ws.p, ws.bytes, s);
    });
  });
}

// problem, weights, x, logits, bias, out, ws, stream
PyObject* forward_few(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run(n, 8, [&] {
    const moe_problem_t p = problem<moe_problem_t>(v[0]);
    const moe_weights_t w = problem<moe_weights_t>(v[1]);
    const int64_t T = p.T;
    void* x = flat(v[2], T * p.H, kBf16, "x");
    void* logits = flat(v[3], T * p.E, kFloat, "logits");
    void* bias = flat(v[4], p.E, kFloat, "bias");
    void* out = flat(v[5], T * p.H, kBf16, "out");
    const Workspace ws(v[6]);
    const moe_stream_t s = stream_of(v[7]);
    return unlocked([&] {
      return moe_forward_few(&p, &w, x, static_cast<float*>(logits), static_cast<float*>(bias), out, ws.p, ws.bytes, s);
    });
  });
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(add_rms_norm), ENTRY(router_logits), ENTRY(gemm_fp8_block), ENTRY(gemm_fp8_block_swiglu),
                         ENTRY(forward_few), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module); }
