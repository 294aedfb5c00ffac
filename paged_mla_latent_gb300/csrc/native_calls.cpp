// The Python calls of the entry points whose kernels take a few microseconds: each torch tensor
// becomes its mla_tensor_t and the C function is called, in one step (13 descriptors cost a
// microsecond so; packed one by one from Python and passed through ctypes, nine).
//
// A call's arguments are the C function's, one for one, after the CUDA device index that its
// tensors must be on: a tensor or None for a descriptor, an int32 tensor for an error word, a
// number for the rest (addresses and streams as integers).  Returns the status.
#include <Python.h>

#include <ATen/core/TensorBase.h>
#include <torch/csrc/autograd/python_variable.h>

#include <tuple>
#include <utility>

#include "../../include/paged_mla.h"

namespace {

constexpr int kMostTensors = 20;

struct Call {
  long device;
  mla_tensor_t tensors[kMostTensors];
  int n = 0;
};

const at::Tensor* tensor_on(PyObject* o, const Call& c) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a torch.Tensor");
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != c.device) {
    PyErr_Format(PyExc_ValueError, "expected a tensor on CUDA device %ld, got one on %s", c.device,
                 t.device().str().c_str());
    return nullptr;
  }
  return &t;
}

template <class T>
struct Arg;

template <>
struct Arg<const mla_tensor_t*> {
  static const mla_tensor_t* from(PyObject* o, Call& c) {
    if (o == Py_None || PyErr_Occurred()) return nullptr;
    const at::Tensor* t = tensor_on(o, c);
    if (!t) return nullptr;
    if (t->dim() > 4) {
      PyErr_SetString(PyExc_ValueError, "at most 4 dimensions");
      return nullptr;
    }
    mla_tensor_t& d = c.tensors[c.n++];
    switch (t->scalar_type()) {
      case at::kByte:                          // raw e4m3fn codes
      case at::kFloat8_e4m3fn: d.dtype = MLA_DTYPE_FP8_E4M3FN; break;
      case at::kBFloat16: d.dtype = MLA_DTYPE_BF16; break;
      case at::kFloat: d.dtype = MLA_DTYPE_FP32; break;
      case at::kInt: d.dtype = MLA_DTYPE_INT32; break;
      default:
        PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t->scalar_type()));
        return nullptr;
    }
    d.ptr = t->mutable_data_ptr();           // (a lazy clone gets its own memory: it may be an output)
    d.ndim = static_cast<int32_t>(t->dim());
    for (int i = 0; i < d.ndim; ++i) {
      d.shape[i] = t->size(i);
      d.stride[i] = t->stride(i);
    }
    for (int i = d.ndim; i < 4; ++i) d.shape[i] = d.stride[i] = 0;
    return &d;
  }
};

template <>
struct Arg<int32_t*> {                         // an error word
  static int32_t* from(PyObject* o, Call& c) {
    if (PyErr_Occurred()) return nullptr;
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.is_cuda() && t.get_device() == c.device && t.scalar_type() == at::kInt && t.numel() >= 1 &&
          t.is_contiguous())
        return static_cast<int32_t*>(t.data_ptr());
    }
    PyErr_Format(PyExc_ValueError, "error_word must be a contiguous int32 tensor on CUDA device %ld", c.device);
    return nullptr;
  }
};

template <>
struct Arg<int32_t> {
  static int32_t from(PyObject* o, Call&) {
    if (PyErr_Occurred()) return 0;
    const long x = PyLong_AsLong(o);
    if (x != static_cast<int32_t>(x)) PyErr_SetString(PyExc_OverflowError, "does not fit 32 bits");
    return static_cast<int32_t>(x);
  }
};

template <>
struct Arg<float> {
  static float from(PyObject* o, Call&) { return PyErr_Occurred() ? 0.f : static_cast<float>(PyFloat_AsDouble(o)); }
};

template <>
struct Arg<size_t> {
  static size_t from(PyObject* o, Call&) { return PyErr_Occurred() ? 0 : PyLong_AsSize_t(o); }
};

template <>
struct Arg<void*> {
  static void* from(PyObject* o, Call&) { return PyErr_Occurred() ? nullptr : PyLong_AsVoidPtr(o); }
};

template <>
struct Arg<mla_stream_t> {
  static mla_stream_t from(PyObject* o, Call&) {
    return PyErr_Occurred() ? nullptr : static_cast<mla_stream_t>(PyLong_AsVoidPtr(o));
  }
};

template <class... A, size_t... I>
PyObject* call_with(int (*fn)(A...), PyObject* const* args, std::index_sequence<I...>) {
  Call c;
  c.device = PyLong_AsLong(args[0]);
  const std::tuple<A...> a{Arg<A>::from(args[I + 1], c)...};     // in their order
  if (PyErr_Occurred()) return nullptr;
  int rc = 0;
  Py_BEGIN_ALLOW_THREADS
  rc = fn(std::get<I>(a)...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

template <class... A>
PyObject* call(int (*fn)(A...), PyObject* const* args, Py_ssize_t n) {
  static_assert(sizeof...(A) <= kMostTensors, "a descriptor each at most");
  if (n != static_cast<Py_ssize_t>(sizeof...(A)) + 1) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", static_cast<int>(sizeof...(A)) + 1, n);
    return nullptr;
  }
  try {
    return call_with(fn, args, std::index_sequence_for<A...>{});
  } catch (const std::exception& e) {          // a tensor without storage or strides
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

template <auto kFn>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(kFn, args, n);
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<&name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(mla_build_page_table), ENTRY(mla_gqa_block_append), ENTRY(mla_gqa_block_gather),
                         ENTRY(mla_gqa_block_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pmla_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pmla_native() { return PyModule_Create(&module); }
