// The operators around the layers from Python: their arguments checked and handed
// to the C entry points, as paged_binding.cpp does for the paged memory.
#include "binding.h"

namespace {

using namespace txl_binding;

// Int32 of any shape, in one piece.
int* ids(const Place& place, const at::Tensor& t) {
  if (t.scalar_type() != at::kInt) throw BadArgument("tokens must be int32");
  return static_cast<int*>(place.of(t));
}

// A dense [.., d] of one row per token.
void* rows(const Place& place, const at::Tensor& t, const at::Tensor& tokens, long long d, const char* name) {
  const bool ok = t.dim() == tokens.dim() + 1 && t.sizes().slice(0, tokens.dim()) == tokens.sizes() &&
                  t.size(tokens.dim()) == d;
  if (!ok) throw BadArgument(std::string(name) + " must be [*tokens.shape, d]");
  return place.of(t);
}

float real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(x);
}

// An fp32 vector of n entries; None: null.
float* reals(const Place& place, PyObject* o, long long n, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != at::kFloat || !shaped(t, {n}))
    throw BadArgument(std::string(name) + " must be fp32 of " + std::to_string(n) + " entries");
  return static_cast<float*>(place.of(t));
}

// (tokens, table, out, scale, stream)
int embed_forward(PyObject* const* a) {
  const at::Tensor &tokens = tensor(a[0]), &table = tensor(a[1]), &out = tensor(a[2]);
  const Place place(tokens);
  if (table.dim() != 2) throw BadArgument("table must be [V, d]");
  return call(txl_embed_forward, ids(place, tokens), place.of(table), rows(place, out, tokens, table.size(1), "out"),
              count(tokens.numel()), count(table.size(0)), count(table.size(1)), real(a[3]), dtype_of(table),
              dtype_of(out), place.stream(a[4]));
}

// (tokens, dout, dtable, scale, accumulate, stream)
int embed_backward(PyObject* const* a) {
  const at::Tensor &tokens = tensor(a[0]), &dout = tensor(a[1]), &dtable = tensor(a[2]);
  const Place place(tokens);
  if (dtable.dim() != 2 || dtable.scalar_type() != at::kFloat) throw BadArgument("dtable must be fp32 [V, d]");
  const int accumulate = PyObject_IsTrue(a[4]);
  if (accumulate < 0) throw PythonError{};
  return call(txl_embed_backward, ids(place, tokens), rows(place, dout, tokens, dtable.size(1), "dout"),
              static_cast<float*>(place.of(dtable)), count(tokens.numel()), count(dtable.size(0)),
              count(dtable.size(1)), real(a[3]), accumulate, dtype_of(dout), place.stream(a[5]));
}

// (x, codes, scales, y, bias, relu, stream)
int dense_w4(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0]), &codes = tensor(a[1]), &scales = tensor(a[2]), &y = tensor(a[3]);
  const Place place(x);
  if (x.dim() != 2 || codes.dim() != 2 || scales.dim() != 2) throw BadArgument("x, codes and scales are matrices");
  const long long m = x.size(0), k = x.size(1), n = codes.size(0), groups = scales.size(0);
  if (k % 2 != 0 || !shaped(codes, {n, k / 2}) || !shaped(scales, {groups, n}) || !shaped(y, {m, n}))
    throw BadArgument("x must be [m, k], codes [n, k / 2], scales [k / group, n], y [m, n]");
  if (x.scalar_type() != at::kBFloat16 || scales.scalar_type() != at::kBFloat16 || codes.scalar_type() != at::kByte)
    throw BadArgument("x and scales must be bf16, codes uint8");
  if (groups <= 0 || k % groups != 0) throw BadArgument("the groups must share k equally");
  const int relu = PyObject_IsTrue(a[5]);
  if (relu < 0) throw PythonError{};
  return call(txl_dense_w4, place.of(x), place.of(codes), place.of(scales), place.of(y), count(m), count(n), count(k),
              count(k / groups), reals(place, a[4], n, "bias"), relu, dtype_of(y), place.stream(a[6]));
}

// (logits, uniform, tokens, temperature, top_k, top_p, min_p, prob, stream)
int sample(PyObject* const* a) {
  const at::Tensor &z = tensor(a[0]), &tokens = tensor(a[2]);
  const Place place(tokens);
  if (z.dim() != 2) throw BadArgument("logits must be [B, V]");
  const long long B = z.size(0), V = z.size(1);
  if (!z.is_cuda() || z.device().index() != place.dev) throw BadArgument(kPlace);
  if ((V > 1 && z.stride(1) != 1) || (B > 1 && z.stride(0) < V)) throw BadArgument("a row's logits must be contiguous");
  if (a[1] == Py_None || a[2] == Py_None) throw BadArgument("uniform and tokens are needed");
  return call(txl_sample, z.data_ptr(), B > 1 ? static_cast<long long>(z.stride(0)) : V, count(B), count(V),
              reals(place, a[1], B, "uniform"), reals(place, a[3], B, "temperature"), place.vector(a[4], B),
              reals(place, a[5], B, "top_p"), reals(place, a[6], B, "min_p"), place.vector(a[2], B),
              reals(place, a[7], B, "prob"), dtype_of(z), place.stream(a[8]));
}

}  // namespace

namespace txl_binding {

PyMethodDef token_methods[] = {method<embed_forward, 5>("embed_forward"), method<embed_backward, 6>("embed_backward"),
                               method<dense_w4, 7>("dense_w4"), method<sample, 9>("sample"),
                               {nullptr, nullptr, 0, nullptr}};

}  // namespace txl_binding
