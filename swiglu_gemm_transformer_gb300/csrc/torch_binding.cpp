// torch_binding.cpp -- the PyTorch side of the sparse MLP block's calls: checks
// of the tensors, outputs, the current stream, and the call of the C ABI.
//
// The block's calls run for a few microseconds at a few tokens, where the same
// marshalling in Python took longer than the kernels (routing one token: 21 us
// of host time a call with ctypes).  A CPython module without pybind11: its
// functions take positional arguments from the wrappers in __init__.py.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <optional>

#include "swiglu.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {};  // a Python error is set

const char *type_name(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    default: return c10::toString(t);
  }
}

template <class... Args>
[[noreturn]] void refuse(PyObject *kind, const char *format, Args... args) {
  PyErr_Format(kind, format, args...);
  throw Refused();
}

// One call: its name, and the device that its tensors share.
struct Call {
  const char *name;
  int device = -1;

  // The tensor argument `o`, of `dims` dimensions, contiguous, on the call's device.
  const Tensor &tensor(PyObject *o, const char *what, int dims, bool rows_only = false) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", what);
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor (there is no CPU path)", what);
    if (device < 0) device = t.get_device();
    if (t.get_device() != device)
      refuse(PyExc_ValueError, "%s: tensors on several devices: cuda:%d, cuda:%d", name, device,
             static_cast<int>(t.get_device()));
    if (!rows_only && (t.dim() != dims || !t.is_contiguous()))
      refuse(PyExc_ValueError, "%s must be a contiguous %d-D tensor", what, dims);
    return t;
  }
  const Tensor &tensor(PyObject *o, const char *what, ScalarType type, int dims) {
    const Tensor &t = tensor(o, what, dims);
    if (t.scalar_type() != type)
      refuse(PyExc_TypeError, "%s must be %s, got %s", what, type_name(type), type_name(t.scalar_type()));
    return t;
  }
  // A tensor that is BF16 or FP32.
  const Tensor &either(PyObject *o, const char *what, int dims) {
    if (THPVariable_Check(o)) {
      const ScalarType t = THPVariable_Unpack(o).scalar_type();
      if (t != ScalarType::BFloat16 && t != ScalarType::Float)
        refuse(PyExc_TypeError, "%s must be bfloat16 or float32, got %s", what, type_name(t));
    }
    return tensor(o, what, dims);
  }
  // An output: the caller's, or a new one.
  Tensor output(PyObject *o, const char *what, ScalarType type, at::IntArrayRef shape) {
    if (o == Py_None)  // from the caching allocator, past the dispatcher (routing one token: 8.4 -> 7.2 us)
      return Tensor(at::detail::empty_cuda(
          shape, type, c10::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)), std::nullopt));
    const Tensor &t = tensor(o, what, type, static_cast<int>(shape.size()));
    if (t.sizes() != shape) {
      if (shape.size() == 1) refuse(PyExc_ValueError, "%s must be [%lld]", what, (long long)shape[0]);
      refuse(PyExc_ValueError, "%s must be [%lld, %lld]", what, (long long)shape[0], (long long)shape[1]);
    }
    return t;
  }
  // Makes the stream argument's stream the current one: None (it is already), a
  // handle, or an object with one.  Outputs and workspaces come from the
  // allocator's pool of the current stream, so memory that work of another
  // stream still uses is not handed to this call, nor this call's to others.
  cudaStream_t enter(PyObject *o, c10::cuda::OptionalCUDAStreamGuard &guard) const {
    const auto dev = static_cast<c10::DeviceIndex>(device);
    const cudaStream_t current = c10::cuda::getCurrentCUDAStream(dev).stream();
    if (o == Py_None) return current;
    PyObject *h = PyLong_Check(o) ? (Py_INCREF(o), o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Refused();
    void *p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Refused();
    const auto s = static_cast<cudaStream_t>(p);
    // (the handle of the legacy default stream has no pool of its own)
    const cudaStream_t pool = s == cudaStreamLegacy ? nullptr : s;
    if (pool != current) guard.reset_stream(c10::cuda::getStreamFromExternal(pool, dev));
    return s;
  }
  // Raises SwigluError for a status other than SWIGLU_OK.
  void check(int status) const {
    if (status == SWIGLU_OK) return;
    PyObject *m = PyImport_ImportModule("swiglu_gemm_transformer_gb300");
    PyObject *cls = m ? PyObject_GetAttrString(m, "SwigluError") : nullptr;
    PyObject *e = cls ? PyObject_CallFunction(cls, "si", name, status) : nullptr;
    if (e) PyErr_SetObject(cls, e);
    Py_XDECREF(e);
    Py_XDECREF(cls);
    Py_XDECREF(m);
    throw Refused();
  }
};

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}

template <class T>
T *ptr(const Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}

// The library call without the interpreter's lock.
template <class F>
int unlocked(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return rc;
}

// Runs `f`, turning C++ exceptions into Python ones.
template <class F>
PyObject *guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (logits, k, renormalize, scale, ids, weights, offsets, rows, slots, workspace, stream)
PyObject *moe_route(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 11) refuse(PyExc_TypeError, "moe_route takes 11 arguments");
    Call c{"swiglu_moe_route"};
    const Tensor &logits = c.either(a[0], "logits", 2);
    const int64_t T = logits.size(0), E = logits.size(1), k = integer(a[1]);
    if (k < 1 || k > E)
      refuse(PyExc_ValueError, "k must be in [1, %lld], got %lld", (long long)E, (long long)k);
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.device));
    c10::cuda::OptionalCUDAStreamGuard pool;
    void *s = c.enter(a[10], pool);
    Tensor out[5] = {c.output(a[4], "ids", ScalarType::Int, {T, k}),
                     c.output(a[5], "weights", ScalarType::Float, {T, k}),
                     c.output(a[6], "offsets", ScalarType::Int, {E + 1}),
                     c.output(a[7], "rows", ScalarType::Int, {T * k}),
                     c.output(a[8], "slots", ScalarType::Int, {T, k})};
    uint64_t bytes = swiglu_moe_route_workspace_size(T, E, k);
    Tensor ws;
    if (a[9] != Py_None) {
      ws = c.tensor(a[9], "workspace", 1);
      bytes = ws.nbytes();
    } else if (bytes > 0) {
      ws = c.output(Py_None, "workspace", ScalarType::Byte, {static_cast<int64_t>(bytes)});
    }
    const bool fp32 = logits.scalar_type() == ScalarType::Float, renorm = truth(a[2]);
    const float scale = static_cast<float>(number(a[3]));
    c.check(unlocked([&] {
      return swiglu_moe_route(logits.data_ptr(), fp32, renorm, scale, ptr<int32_t>(out[0]),
                              ptr<float>(out[1]), ptr<int32_t>(out[2]), ptr<int32_t>(out[3]),
                              ptr<int32_t>(out[4]), T, E, k, ws.defined() ? ws.data_ptr() : nullptr, bytes, s);
    }));
    PyObject *r = PyTuple_New(5);
    if (!r) throw Refused();
    for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(out[i])));
    return r;
  });
}

// (A, W1, W2 or None, offsets, rows or None, Y or None, stream)
PyObject *grouped(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 7) refuse(PyExc_TypeError, "grouped takes 7 arguments");
    const bool fused = a[2] != Py_None;
    Call c{fused ? "swiglu_fused_grouped" : "swiglu_linear_grouped"};
    const Tensor &A = c.tensor(a[0], fused ? "A" : "X", ScalarType::BFloat16, 2);
    const Tensor &W1 = c.tensor(a[1], fused ? "W1" : "W", ScalarType::BFloat16, 3);
    const Tensor &W2 = fused ? c.tensor(a[2], "W2", ScalarType::BFloat16, 3) : W1;
    if (W2.sizes() != W1.sizes()) refuse(PyExc_ValueError, "W1 and W2 must match in shape");
    const int64_t T = A.size(0), K = A.size(1), E = W1.size(0), N = W1.size(2);
    if (W1.size(1) != K)
      refuse(PyExc_ValueError, "shape mismatch: rows of %lld, weights [%lld, %lld, %lld]", (long long)K,
             (long long)E, (long long)W1.size(1), (long long)N);
    const Tensor &offsets = c.tensor(a[3], "offsets", ScalarType::Int, 1);
    if (offsets.numel() != E + 1) refuse(PyExc_ValueError, "offsets must have %lld elements", (long long)E + 1);
    const Tensor *rows = a[4] != Py_None ? &c.tensor(a[4], "rows", ScalarType::Int, 1) : nullptr;
    const int64_t P = rows ? rows->numel() : T;
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.device));
    c10::cuda::OptionalCUDAStreamGuard pool;
    void *s = c.enter(a[6], pool);
    Tensor Y = c.output(a[5], "the output", ScalarType::BFloat16, {P, N});
    // (an empty tensor has no address: any other stands for "rows are given")
    const int32_t *r = !rows ? nullptr : P > 0 ? ptr<int32_t>(*rows) : ptr<int32_t>(offsets);
    c.check(unlocked([&] {
      return fused ? swiglu_fused_grouped(A.data_ptr(), W1.data_ptr(), W2.data_ptr(), ptr<int32_t>(offsets),
                                          r, Y.data_ptr(), T, P, E, N, K, s)
                   : swiglu_linear_grouped(A.data_ptr(), W1.data_ptr(), ptr<int32_t>(offsets), r,
                                           Y.data_ptr(), T, P, E, N, K, s);
    }));
    return THPVariable_Wrap(std::move(Y));
  });
}

// (Z, R, slots, weights, post_norm, gamma_post, gate, residual_scale, pre_norm, gamma_pre, eps, Rout, H, stream)
PyObject *residual_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 14) refuse(PyExc_TypeError, "residual_norm takes 14 arguments");
    Call c{"swiglu_residual_norm"};
    const auto bf = ScalarType::BFloat16;
    const Tensor &Z = c.tensor(a[0], "Z", bf, 2);
    const Tensor &R = c.either(a[1], "R", 2);
    const int64_t T = R.size(0), D = R.size(1), P = Z.size(0);
    if (Z.size(1) != D)
      refuse(PyExc_ValueError, "shape mismatch: Z [%lld, %lld], R [%lld, %lld]", (long long)P,
             (long long)Z.size(1), (long long)T, (long long)D);
    if ((a[2] == Py_None) != (a[3] == Py_None)) refuse(PyExc_ValueError, "slots and weights go together");
    const Tensor *slots = nullptr, *weights = nullptr;
    int64_t k = 0;
    if (a[2] == Py_None) {
      if (P != T) refuse(PyExc_ValueError, "without slots, Z must be [T, D]");
    } else {
      slots = &c.tensor(a[2], "slots", ScalarType::Int, 2);
      weights = &c.tensor(a[3], "weights", ScalarType::Float, 2);
      k = slots->size(1);
      if (slots->size(0) != T || weights->size(0) != T || weights->size(1) != k)
        refuse(PyExc_ValueError, "slots and weights must be [T, k]");
    }
    const bool post = truth(a[4]), pre = truth(a[8]);
    const Tensor *gamma[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
      PyObject *o = a[i == 0 ? 5 : 9];
      if (o == Py_None) continue;
      const char *what = i == 0 ? "gamma_post" : "gamma_pre";
      gamma[i] = &c.tensor(o, what, bf, 1);
      if (gamma[i]->numel() != D) refuse(PyExc_ValueError, "%s must have %lld elements", what, (long long)D);
    }
    if (gamma[0] && !post) refuse(PyExc_ValueError, "gamma_post without post_norm");
    if (gamma[1] && !pre) refuse(PyExc_ValueError, "gamma_pre without pre_norm");
    if (a[12] != Py_None && !pre) refuse(PyExc_ValueError, "H without pre_norm");
    const Tensor *gate = nullptr;
    int64_t stride = 0;
    if (a[6] != Py_None) {
      gate = &c.tensor(a[6], "gate", 0, true);
      if (gate->scalar_type() != bf)
        refuse(PyExc_TypeError, "gate must be %s, got %s", type_name(bf), type_name(gate->scalar_type()));
      const bool shape = gate->dim() == 1 ? gate->size(0) == D
                                          : gate->dim() == 2 && gate->size(0) == T && gate->size(1) == D;
      if (!shape || (D > 1 && gate->stride(gate->dim() - 1) != 1))
        refuse(PyExc_ValueError, "gate must be [D] or [T, D] with contiguous rows");
      stride = gate->dim() == 2 && T > 1 ? gate->stride(0) : 0;
    }
    const float scale = static_cast<float>(number(a[7])), eps = static_cast<float>(number(a[10]));
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.device));
    c10::cuda::OptionalCUDAStreamGuard pool;
    void *s = c.enter(a[13], pool);
    Tensor Rout = c.output(a[11], "Rout", R.scalar_type(), {T, D});
    Tensor H;
    if (pre) H = c.output(a[12], "H", bf, {T, D});
    // (slots without columns have no address: any other stands for "slots are given")
    auto at = [&](const Tensor *t) { return !t ? nullptr : t->numel() > 0 ? t->data_ptr() : R.data_ptr(); };
    c.check(unlocked([&] {
      return swiglu_residual_norm(Z.data_ptr(), static_cast<const int32_t *>(at(slots)),
                                  static_cast<const float *>(at(weights)), R.data_ptr(),
                                  R.scalar_type() == ScalarType::Float, post, at(gamma[0]), at(gate), stride,
                                  scale, at(gamma[1]), eps, Rout.data_ptr(), pre ? H.data_ptr() : nullptr, T, P, k, D, s);
    }));
    PyObject *r = PyTuple_New(2);
    if (!r) throw Refused();
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(Rout)));
    // (an undefined tensor is None)
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(H)));
    return r;
  });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"moe_route", fast<moe_route>(), METH_FASTCALL, nullptr},
    {"grouped", fast<grouped>(), METH_FASTCALL, nullptr},
    {"residual_norm", fast<residual_norm>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_swiglu_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__swiglu_torch(void) { return PyModule_Create(&module); }
