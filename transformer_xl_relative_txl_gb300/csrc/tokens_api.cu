// C entry points of the operators around the layers (see
// include/txl_relattn.h): argument checks, alias checks, dispatch.
#include <cmath>
#include <cstdint>

#include "tokens.h"
#include "txl_internal.h"
#include "txl_relattn.h"

namespace {

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
Range range_of(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, p == nullptr ? a : a + bytes};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }
template <typename... R>
bool overlaps_any(Range a, R... b) {
  return (overlap(a, b) || ...);
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool type_ok(int t) { return t == TXL_F32 || t == TXL_BF16; }
size_t size_of(int t) { return t == TXL_BF16 ? 2 : 4; }
size_t times(long long a, long long b, size_t c) { return static_cast<size_t>(a) * static_cast<size_t>(b) * c; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? TXL_OK : TXL_ERR_CUDA; }

constexpr int kMaxTokens = 1 << 30, kMaxWidth = 1 << 20;

}  // namespace

extern "C" {

int txl_embed_forward(const int* tokens, const void* table, void* out, int T, int V, int d, float scale,
                      txl_dtype table_dtype, txl_dtype out_dtype, cudaStream_t stream) {
  if (T < 0 || V <= 0 || d <= 0 || !type_ok(table_dtype) || !type_ok(out_dtype)) return TXL_ERR_INVALID_ARG;
  if (T == 0) return TXL_OK;
  if (T > kMaxTokens || V > txl::kEmbedMaxRows || d > kMaxWidth) return TXL_ERR_UNSUPPORTED;
  if (tokens == nullptr || table == nullptr || out == nullptr || !aligned(tokens, 4) ||
      !aligned(table, size_of(table_dtype)) || !aligned(out, size_of(out_dtype)))
    return TXL_ERR_INVALID_ARG;
  if (overlaps_any(range_of(out, times(T, d, size_of(out_dtype))), range_of(tokens, times(T, 1, 4)),
                   range_of(table, times(V, d, size_of(table_dtype)))))
    return TXL_ERR_ALIAS;
  return from_cuda(txl::launch_embed_forward(tokens, table, out, T, V, d, scale, table_dtype == TXL_BF16,
                                             out_dtype == TXL_BF16, stream));
}

int txl_embed_backward(const int* tokens, const void* dout, float* dtable, int T, int V, int d, float scale,
                       int accumulate, txl_dtype dtype, cudaStream_t stream) {
  if (T < 0 || V <= 0 || d <= 0 || !type_ok(dtype)) return TXL_ERR_INVALID_ARG;
  if (T == 0 && accumulate != 0) return TXL_OK;
  if (T > kMaxTokens || V > txl::kEmbedMaxRows || d > kMaxWidth) return TXL_ERR_UNSUPPORTED;
  if (dtable == nullptr || !aligned(dtable, 4)) return TXL_ERR_INVALID_ARG;
  if (T > 0 && (tokens == nullptr || dout == nullptr || !aligned(tokens, 4) || !aligned(dout, size_of(dtype))))
    return TXL_ERR_INVALID_ARG;
  if (T > 0 && overlaps_any(range_of(dtable, times(V, d, 4)), range_of(tokens, times(T, 1, 4)),
                            range_of(dout, times(T, d, size_of(dtype)))))
    return TXL_ERR_ALIAS;
  return from_cuda(txl::launch_embed_backward(tokens, dout, dtable, T, V, d, scale, accumulate != 0,
                                              dtype == TXL_BF16, stream));
}

int txl_dense_w4(const void* x, const void* codes, const void* scales, void* y, int m, int n, int k, int group,
                 const float* bias, int relu, txl_dtype y_dtype, cudaStream_t stream) {
  if (m < 0 || n <= 0 || k <= 0 || !type_ok(y_dtype)) return TXL_ERR_INVALID_ARG;
  if (m == 0) return TXL_OK;
  if ((group != 32 && group != 64 && group != 128) || k % group != 0 || n % 8 != 0 || m > kMaxWidth ||
      n > (1 << 30) || k > (1 << 24))
    return TXL_ERR_UNSUPPORTED;
  if (x == nullptr || codes == nullptr || scales == nullptr || y == nullptr || !aligned(x, 16) ||
      !aligned(codes, 16) || !aligned(scales, 16) || !aligned(y, size_of(y_dtype)) || !aligned(bias, 4))
    return TXL_ERR_INVALID_ARG;
  if (overlaps_any(range_of(y, times(m, n, size_of(y_dtype))), range_of(x, times(m, k, 2)),
                   range_of(codes, times(n, k / 2, 1)), range_of(scales, times(k / group, n, 2)),
                   range_of(bias, times(n, 1, 4))))
    return TXL_ERR_ALIAS;
  return from_cuda(txl::launch_dense_w4(x, static_cast<const unsigned char*>(codes), scales, y, bias, m, n, k, group,
                                        relu != 0, y_dtype == TXL_BF16, stream));
}

int txl_sample(const void* logits, long long row_stride, int B, int V, const float* uniform,
               const float* temperature, const int* top_k, const float* top_p, const float* min_p, int* tokens,
               float* prob, txl_dtype dtype, cudaStream_t stream) {
  if (B < 0 || V <= 0 || !type_ok(dtype) || (B > 1 && row_stride < V)) return TXL_ERR_INVALID_ARG;
  if (B == 0) return TXL_OK;
  if (V > txl::kSampleMaxVocab || B > 65535 || row_stride > (1LL << 40)) return TXL_ERR_UNSUPPORTED;
  if (logits == nullptr || uniform == nullptr || tokens == nullptr || !aligned(logits, size_of(dtype)))
    return TXL_ERR_INVALID_ARG;
  const void* const words[] = {uniform, temperature, top_k, top_p, min_p, tokens, prob};
  for (const void* p : words)
    if (!aligned(p, 4)) return TXL_ERR_INVALID_ARG;
  const size_t vec = times(B, 1, 4);
  const Range z = range_of(logits, (times(B - 1, B > 1 ? row_stride : 0, 1) + V) * size_of(dtype));
  const Range out = range_of(tokens, vec), pr = range_of(prob, vec);
  if (overlap(out, pr)) return TXL_ERR_ALIAS;
  for (const Range& r : {out, pr})
    if (overlaps_any(r, z, range_of(uniform, vec), range_of(temperature, vec), range_of(top_k, vec),
                     range_of(top_p, vec), range_of(min_p, vec)))
      return TXL_ERR_ALIAS;
  const txl::SampleArgs a{logits, row_stride, B,     V,      uniform, temperature,
                          top_k,  top_p,      min_p, tokens, prob,    dtype == TXL_BF16};
  return from_cuda(txl::launch_sample(a, stream));
}

}  // extern "C"
