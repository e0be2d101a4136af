// The paged memory's calls from Python: torch tensors checked and handed to
// the C entry points, one call of this module for one of theirs.  The package's
// functions of the same names pass their arguments on and raise for a status
// that is not 0.
//
// A token's step is three or four such calls of 3 to 10 us on the GPU, each
// with up to 14 tensors.  Checked from Python (dtype, shape, device, pointer of
// each) a call took 9 us on the host, and the host was what a step took; here
// it takes 2, most of it the launch.
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

namespace {

struct BadArgument : std::runtime_error {  // ValueError
  using std::runtime_error::runtime_error;
};
struct PythonError {};  // already set

const char* const kPlace = "tensors must live in the current device's memory";

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a tensor");
    throw PythonError{};
  }
  return THPVariable_Unpack(o);
}

int integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PythonError{};
  if (x < std::numeric_limits<int>::min() || x > std::numeric_limits<int>::max())
    throw BadArgument("an integer past 32 bits");
  return static_cast<int>(x);
}

int count(long long n) {
  if (n > std::numeric_limits<int>::max()) throw BadArgument("more than 2^31 - 1 entries");
  return static_cast<int>(n);
}

bool shaped(const at::Tensor& t, std::initializer_list<long long> shape) {
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

txl_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return TXL_BF16;
  if (t.scalar_type() == at::kFloat) return TXL_F32;
  throw BadArgument(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}

// A page book: a dict of int32 tensors table [slots, max_pages], start and rows
// [slots], refs [pages].
txl_page_book book_of(const Place& at_, PyObject* book, int page_rows) {
  static PyObject* const names[4] = {PyUnicode_InternFromString("table"), PyUnicode_InternFromString("start"),
                                     PyUnicode_InternFromString("rows"), PyUnicode_InternFromString("refs")};
  const at::Tensor* t[4];
  if (!PyDict_Check(book)) {
    PyErr_SetString(PyExc_TypeError, "a book is a dict of tensors");
    throw PythonError{};
  }
  for (int i = 0; i < 4; ++i) {
    PyObject* item = PyDict_GetItemWithError(book, names[i]);
    if (item == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetObject(PyExc_KeyError, names[i]);
      throw PythonError{};
    }
    t[i] = &tensor(item);
  }
  if (t[0]->dim() != 2 || !shaped(*t[1], {t[0]->size(0)}) || !shaped(*t[2], {t[0]->size(0)}) || t[3]->dim() != 1)
    throw BadArgument("a book is table [slots, max_pages], start and rows [slots], refs [pages]");
  for (const at::Tensor* x : t)
    if (x->scalar_type() != at::kInt) throw BadArgument("a book's tensors are int32");
  txl_page_book b{};
  b.table = static_cast<int*>(at_.of(*t[0]));
  b.start = static_cast<int*>(at_.of(*t[1]));
  b.rows = static_cast<int*>(at_.of(*t[2]));
  b.refs = static_cast<int*>(at_.of(*t[3]));
  b.n_slots = count(t[0]->size(0));
  b.max_pages = count(t[0]->size(1));
  b.n_pages = count(t[3]->size(0));
  b.page_rows = page_rows;
  return b;
}

// The pools [pages, H, page_rows, D].
struct Pools {
  const at::Tensor &kt, &vt;
  void *k, *v;
  int pages, H, page_rows, D;
  txl_dtype dtype;
  Pools(const Place& place, PyObject* ko, PyObject* vo) : kt(tensor(ko)), vt(tensor(vo)) {
    if (kt.dim() != 4 || vt.sizes() != kt.sizes() || vt.scalar_type() != kt.scalar_type())
      throw BadArgument("k_pages, v_pages must be [pages, H, page_rows, D] of one dtype");
    k = place.of(kt);
    v = place.of(vt);
    pages = count(kt.size(0));
    H = count(kt.size(1));
    page_rows = count(kt.size(2));
    D = count(kt.size(3));
    dtype = dtype_of(kt);
  }
  void of(const txl_page_book& b) const {
    if (b.n_pages != pages) throw BadArgument("the pools' pages must be those that refs counts");
  }
};

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

// (book, page_rows, slots, cu, granted, copy_src, copy_dst, stream)
int reserve(PyObject* const* a) {
  const at::Tensor& slots = tensor(a[2]);
  const Place place(slots);
  const long long n = slots.numel();
  const txl_page_book b = book_of(place, a[0], integer(a[1]));
  return call(txl_pages_reserve, &b, place.vector(a[2], n), place.vector(a[3], n + 1), count(n), place.vector(a[4], n),
              place.vector(a[5], n), place.vector(a[6], n), place.stream(a[7]));
}

// (book, k_pages, v_pages, slots, cu, granted, copy_src, copy_dst, k_new, v_new, stream)
int append(PyObject* const* a) {
  const at::Tensor& slots = tensor(a[3]);
  const Place place(slots);
  const long long n = slots.numel();
  const Pools pools(place, a[1], a[2]);
  const txl_page_book b = book_of(place, a[0], pools.page_rows);
  pools.of(b);
  if ((a[6] == Py_None) != (a[7] == Py_None)) throw BadArgument("copy_src and copy_dst come together");
  const at::Tensor &k = tensor(a[8]), &v = tensor(a[9]);
  const long long T = k.dim() == 3 ? k.size(0) : -1;
  if (!shaped(k, {T, pools.H, pools.D}) || !shaped(v, {T, pools.H, pools.D}))
    throw BadArgument("k_new, v_new must be [T, H, D]");
  if (k.scalar_type() != pools.kt.scalar_type() || v.scalar_type() != pools.kt.scalar_type())
    throw BadArgument("the pools and the new rows share a dtype");
  return call(txl_pages_append, &b, pools.k, pools.v, pools.H, pools.D, place.vector(a[3], n),
              place.vector(a[4], n + 1), count(n), place.vector(a[5], n), place.vector(a[6], n), place.vector(a[7], n),
              place.of(k), place.of(v), count(T), pools.dtype, place.stream(a[10]));
}

// (k_pages, v_pages, src, dst, stream)
int copy(PyObject* const* a) {
  const at::Tensor& src = tensor(a[2]);
  const Place place(src);
  const long long n = src.numel();
  const Pools pools(place, a[0], a[1]);
  return call(txl_pages_copy, pools.k, pools.v, pools.pages,
              static_cast<long long>(pools.H) * pools.page_rows * pools.D, place.vector(a[2], n), place.vector(a[3], n),
              count(n), pools.dtype, place.stream(a[4]));
}

// (book, page_rows, src, dst, ok, stream)
int fork(PyObject* const* a) {
  const at::Tensor& src = tensor(a[2]);
  const Place place(src);
  const long long n = src.numel();
  const txl_page_book b = book_of(place, a[0], integer(a[1]));
  return call(txl_pages_fork, &b, place.vector(a[2], n), place.vector(a[3], n), count(n), place.vector(a[4], n),
              place.stream(a[5]));
}

// (book, page_rows, slots, keep, stream)
int free_(PyObject* const* a) {
  const at::Tensor& slots = tensor(a[2]);
  const Place place(slots);
  const long long n = slots.numel();
  const txl_page_book b = book_of(place, a[0], integer(a[1]));
  return call(txl_pages_free, &b, place.vector(a[2], n), place.vector(a[3], n), count(n), place.stream(a[4]));
}

// (book, page_rows, new_id, copy_src, copy_dst, count, stream)
int compact(PyObject* const* a) {
  const Place place(tensor(a[2]));
  const txl_page_book b = book_of(place, a[0], integer(a[1]));
  return call(txl_pages_compact, &b, place.vector(a[2], b.n_pages), place.vector(a[3], b.n_pages),
              place.vector(a[4], b.n_pages), place.vector(a[5], 1), place.stream(a[6]));
}

// (q, k_pages, v_pages, book, slots, cu, r, bias_u, bias_v, o, workspace, lse, max_new, scale, stream)
int attend(PyObject* const* a) {
  const at::Tensor& slots = tensor(a[4]);
  const Place place(slots);
  const long long n = slots.numel();
  const Pools pools(place, a[1], a[2]);
  const txl_page_book b = book_of(place, a[3], pools.page_rows);
  pools.of(b);
  const at::Tensor &q = tensor(a[0]), &r = tensor(a[6]), &u = tensor(a[7]), &v = tensor(a[8]), &o = tensor(a[9]),
                   &ws = tensor(a[10]);
  const int H = pools.H, D = pools.D;
  const long long T = q.dim() == 3 ? q.size(0) : -1, n_r = r.dim() == 3 ? r.size(0) : -1;
  if (!shaped(q, {T, H, D}) || !shaped(o, {T, H, D})) throw BadArgument("q and o must be [T, H, D]");
  if (!shaped(r, {n_r, H, D}) || !shaped(u, {H, D}) || !shaped(v, {H, D}))
    throw BadArgument("r must be [n_r, H, D]; biases [H, D]");
  if (u.scalar_type() != at::kFloat || v.scalar_type() != at::kFloat) throw BadArgument("biases are fp32");
  if (q.scalar_type() != pools.kt.scalar_type() || r.scalar_type() != pools.kt.scalar_type())
    throw BadArgument("q, the pools and r share a dtype");
  float* lse = nullptr;
  if (a[11] != Py_None) {
    const at::Tensor& l = tensor(a[11]);
    if (!shaped(l, {H, T}) || l.scalar_type() != at::kFloat) throw BadArgument("lse must be fp32 [H, T]");
    lse = static_cast<float*>(place.of(l));
  }
  const int most = a[12] == Py_None ? count(T) : integer(a[12]);
  const double scale = PyFloat_AsDouble(a[13]);
  if (scale == -1.0 && PyErr_Occurred()) throw PythonError{};
  return call(txl_relattn_forward_paged, place.of(q), pools.k, pools.v, &b, place.vector(a[4], n),
              place.vector(a[5], n + 1), count(n), count(T), most, place.of(r), static_cast<float*>(place.of(u)),
              static_cast<float*>(place.of(v)), place.of(o), lse, H, D, count(n_r), static_cast<float>(scale),
              pools.dtype, dtype_of(o), place.of(ws), ws.nbytes(), place.stream(a[14]));
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

PyMethodDef methods[] = {method<reserve, 8>("pages_reserve"), method<append, 11>("pages_append"),
                         method<copy, 5>("pages_copy"),       method<fork, 6>("pages_fork"),
                         method<free_, 5>("pages_free"),      method<compact, 7>("pages_compact"),
                         method<attend, 15>("forward_paged"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", "The paged memory's calls on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
