// What the extension module's sources share: torch tensors checked and handed to
// the C entry points, their errors as Python's.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <limits>
#include <stdexcept>
#include <string>

#include "txl_relattn.h"

namespace txl_binding {

struct BadArgument : std::runtime_error {  // ValueError
  using std::runtime_error::runtime_error;
};
struct PythonError {};  // already set

inline const char* const kPlace = "tensors must live in the current device's memory";

inline const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a tensor");
    throw PythonError{};
  }
  return THPVariable_Unpack(o);
}

inline int integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PythonError{};
  if (x < std::numeric_limits<int>::min() || x > std::numeric_limits<int>::max())
    throw BadArgument("an integer past 32 bits");
  return static_cast<int>(x);
}

inline int count(long long n) {
  if (n > std::numeric_limits<int>::max()) throw BadArgument("more than 2^31 - 1 entries");
  return static_cast<int>(n);
}

inline bool shaped(const at::Tensor& t, std::initializer_list<long long> shape) {
  return t.sizes() == c10::IntArrayRef(reinterpret_cast<const int64_t*>(shape.begin()), shape.size());
}
static_assert(sizeof(long long) == sizeof(int64_t), "shapes");

// The device that a call launches on: the current one, where its tensors must
// live.
struct Place {
  int dev;
  explicit Place(const at::Tensor& t) : dev(t.is_cuda() ? t.device().index() : -1) {
    if (dev < 0 || dev != c10::cuda::current_device()) throw BadArgument(kPlace);
  }
  void* of(const at::Tensor& t) const {
    if (!t.is_contiguous()) throw BadArgument("tensors must be contiguous");
    if (!t.is_cuda() || t.device().index() != dev) throw BadArgument(kPlace);
    return t.data_ptr();
  }
  // An int32 vector of n entries; None: null.
  int* vector(PyObject* o, long long n) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != at::kInt || !shaped(t, {n}) || !t.is_contiguous())
      throw BadArgument("expected a contiguous int32 vector of " + std::to_string(n) + " entries");
    return static_cast<int*>(of(t));
  }
  cudaStream_t stream(PyObject* o) const {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw PythonError{};
    return static_cast<cudaStream_t>(p);
  }
};

inline txl_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return TXL_BF16;
  if (t.scalar_type() == at::kFloat) return TXL_F32;
  throw BadArgument(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}

// Entry point f on arguments that are made with the interpreter's lock held, run
// without it: a launch waits where the device's queue is full.
template <typename... P, typename... A>
int call(int (*f)(P...), A... args) {
  struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
  } unlocked;
  return f(args...);
}

// The status of call F with its N arguments.
template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const PythonError&) {
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <int (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

// The module's methods of one source each, ended by a method without a name.
extern PyMethodDef token_methods[];

}  // namespace txl_binding
