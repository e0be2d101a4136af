// C entry points of the paged memory (see include/txl_relattn.h): argument
// checks, alias checks, dispatch.
#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"
#include "pages.h"
#include "txl_relattn.h"

namespace {

using txl::PageBook;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
Range range_of(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, p == nullptr ? a : a + bytes};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// Whether any of outs overlaps another of them or one of ins.
template <size_t NO, size_t NI>
bool aliased(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (size_t x = 0; x < NO; ++x) {
    for (const Range& y : ins)
      if (overlap(outs[x], y)) return true;
    for (size_t z = x + 1; z < NO; ++z)
      if (overlap(outs[x], outs[z])) return true;
  }
  return false;
}

size_t ints(long long n) { return static_cast<size_t>(n) * sizeof(int); }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? TXL_OK : TXL_ERR_CUDA; }
bool type_ok(int t) { return t == TXL_F32 || t == TXL_BF16; }
size_t size_of(int t) { return t == TXL_BF16 ? 2 : 4; }

template <typename... P>
bool pointers_ok(size_t align, const P*... p) {
  return ((p != nullptr && aligned(p, align)) && ...);
}

// The ranges of the book's parts (refs empty where the call does not use it).
struct BookRanges {
  Range r[4];
};
BookRanges ranges(const PageBook& b) {
  return {{range_of(b.table, ints(static_cast<long long>(b.n_slots) * b.max_pages)), range_of(b.start, ints(b.n_slots)),
           range_of(b.rows, ints(b.n_slots)), range_of(b.refs, ints(b.n_pages))}};
}

// The book's pointers, sizes and limits; refs: the call uses them.
int check_book(const txl_page_book* p, bool refs, PageBook* out) {
  if (p == nullptr || !pointers_ok(4, p->table, p->start, p->rows) || (refs && !pointers_ok(4, p->refs)))
    return TXL_ERR_INVALID_ARG;
  if (p->n_slots <= 0 || p->max_pages <= 0 || p->n_pages <= 0 || p->page_rows <= 0) return TXL_ERR_INVALID_ARG;
  if ((p->page_rows & (p->page_rows - 1)) != 0 || p->page_rows < 16 || p->page_rows > 1024 ||
      p->n_slots > txl::kMaxSlots || p->n_pages > (1 << 28) ||
      static_cast<long long>(p->max_pages) * p->page_rows > (1 << 30))
    return TXL_ERR_UNSUPPORTED;
  *out = PageBook{p->table,   p->start,     p->rows,    refs ? p->refs : nullptr,
                  p->n_slots, p->max_pages, p->n_pages, p->page_rows};
  const Range none[] = {Range{0, 0}};
  return aliased(ranges(*out).r, none) ? TXL_ERR_ALIAS : TXL_OK;
}

int status_word(unsigned int** status) {
  txl::WaitCtl wc;
  const int rc = txl::api_wait_ctl(&wc);
  *status = wc.status;
  return rc;
}

}  // namespace

extern "C" {

int txl_pages_reserve(const txl_page_book* book, const int* slots, const int* cu, int n, int* granted,
                      int* copy_src, int* copy_dst, cudaStream_t stream) {
  PageBook b;
  if (const int rc = check_book(book, true, &b); rc != TXL_OK) return rc;
  if (n < 0) return TXL_ERR_INVALID_ARG;
  if (n == 0) return TXL_OK;
  if (n > txl::kMaxSlots) return TXL_ERR_UNSUPPORTED;
  if (!pointers_ok(4, slots, cu, granted, copy_src, copy_dst)) return TXL_ERR_INVALID_ARG;
  const BookRanges br = ranges(b);
  const Range outs[] = {range_of(granted, ints(n)), range_of(copy_src, ints(n)), range_of(copy_dst, ints(n)),
                        br.r[0], br.r[1], br.r[2], br.r[3]};
  const Range ins[] = {range_of(slots, ints(n)), range_of(cu, ints(n + 1LL))};
  if (aliased(outs, ins)) return TXL_ERR_ALIAS;
  unsigned int* status;
  if (status_word(&status) != TXL_OK) return TXL_ERR_CUDA;
  return from_cuda(txl::launch_pages_reserve(b, slots, cu, n, granted, copy_src, copy_dst, status, stream));
}

int txl_pages_append(const txl_page_book* book, void* k_pages, void* v_pages, int H, int D, const int* slots,
                     const int* cu, int n, const int* granted, const int* copy_src, const int* copy_dst,
                     const void* k_new, const void* v_new, int T, txl_dtype dtype, cudaStream_t stream) {
  PageBook b;
  if (const int rc = check_book(book, false, &b); rc != TXL_OK) return rc;
  if (n < 0 || T < 0 || H <= 0 || D <= 0 || !type_ok(dtype)) return TXL_ERR_INVALID_ARG;
  if (n == 0 || T == 0) return TXL_OK;
  if (n > txl::kMaxSlots || D > 256 || H > 65535) return TXL_ERR_UNSUPPORTED;
  const size_t es = size_of(dtype);
  if (!pointers_ok(es, static_cast<const char*>(k_pages), static_cast<const char*>(v_pages),
                   static_cast<const char*>(k_new), static_cast<const char*>(v_new)) ||
      !pointers_ok(4, slots, cu, granted))
    return TXL_ERR_INVALID_ARG;
  if ((copy_src == nullptr) != (copy_dst == nullptr) || !aligned(copy_src, 4) || !aligned(copy_dst, 4))
    return TXL_ERR_INVALID_ARG;
  const size_t pool = static_cast<size_t>(b.n_pages) * H * b.page_rows * D * es;
  const size_t rows = static_cast<size_t>(T) * H * D * es;
  const BookRanges br = ranges(b);
  const Range outs[] = {range_of(k_pages, pool), range_of(v_pages, pool)};
  const Range ins[] = {range_of(k_new, rows), range_of(v_new, rows), range_of(slots, ints(n)),
                       range_of(cu, ints(n + 1LL)), range_of(granted, ints(n)), range_of(copy_src, ints(n)),
                       range_of(copy_dst, ints(n)), br.r[0], br.r[1], br.r[2]};
  if (aliased(outs, ins)) return TXL_ERR_ALIAS;
  unsigned int* status;
  if (status_word(&status) != TXL_OK) return TXL_ERR_CUDA;
  return from_cuda(txl::launch_pages_append(b, k_pages, v_pages, H, D, static_cast<int>(es), slots, cu, n, granted,
                                            copy_src, copy_dst, k_new, v_new, T, status, stream));
}

int txl_pages_copy(void* k_pages, void* v_pages, int n_pages, long long page_elems, const int* src, const int* dst,
                   int n, txl_dtype dtype, cudaStream_t stream) {
  if (n < 0 || n_pages <= 0 || page_elems <= 0 || !type_ok(dtype)) return TXL_ERR_INVALID_ARG;
  if (n == 0) return TXL_OK;
  if (n_pages > (1 << 28) || n > (1 << 28) || page_elems > (1LL << 32)) return TXL_ERR_UNSUPPORTED;
  const size_t es = size_of(dtype);
  if (!pointers_ok(es, static_cast<const char*>(k_pages), static_cast<const char*>(v_pages)) ||
      !pointers_ok(4, src, dst))
    return TXL_ERR_INVALID_ARG;
  const size_t pool = static_cast<size_t>(n_pages) * page_elems * es;
  const Range outs[] = {range_of(k_pages, pool), range_of(v_pages, pool)};
  const Range ins[] = {range_of(src, ints(n)), range_of(dst, ints(n))};
  if (aliased(outs, ins)) return TXL_ERR_ALIAS;
  unsigned int* status;
  if (status_word(&status) != TXL_OK) return TXL_ERR_CUDA;
  return from_cuda(txl::launch_pages_copy(k_pages, v_pages, n_pages, page_elems * static_cast<long long>(es), src,
                                          dst, n, status, stream));
}

int txl_pages_fork(const txl_page_book* book, const int* src, const int* dst, int n, int* ok, cudaStream_t stream) {
  PageBook b;
  if (const int rc = check_book(book, true, &b); rc != TXL_OK) return rc;
  if (n < 0) return TXL_ERR_INVALID_ARG;
  if (n == 0) return TXL_OK;
  if (n > txl::kMaxSlots) return TXL_ERR_UNSUPPORTED;
  if (!pointers_ok(4, src, dst, ok)) return TXL_ERR_INVALID_ARG;
  const BookRanges br = ranges(b);
  const Range outs[] = {range_of(ok, ints(n)), br.r[0], br.r[1], br.r[2], br.r[3]};
  const Range ins[] = {range_of(src, ints(n)), range_of(dst, ints(n))};
  if (aliased(outs, ins)) return TXL_ERR_ALIAS;
  unsigned int* status;
  if (status_word(&status) != TXL_OK) return TXL_ERR_CUDA;
  return from_cuda(txl::launch_pages_fork(b, src, dst, n, ok, status, stream));
}

int txl_pages_free(const txl_page_book* book, const int* slots, const int* keep, int n, cudaStream_t stream) {
  PageBook b;
  if (const int rc = check_book(book, true, &b); rc != TXL_OK) return rc;
  if (n < 0) return TXL_ERR_INVALID_ARG;
  if (n == 0) return TXL_OK;
  if (n > txl::kMaxSlots) return TXL_ERR_UNSUPPORTED;
  if (!pointers_ok(4, slots) || !aligned(keep, 4)) return TXL_ERR_INVALID_ARG;
  const BookRanges br = ranges(b);
  const Range ins[] = {range_of(slots, ints(n)), range_of(keep, ints(n))};
  if (aliased(br.r, ins)) return TXL_ERR_ALIAS;
  unsigned int* status;
  if (status_word(&status) != TXL_OK) return TXL_ERR_CUDA;
  return from_cuda(txl::launch_pages_free(b, slots, keep, n, status, stream));
}

int txl_pages_compact(const txl_page_book* book, int* new_id, int* copy_src, int* copy_dst, int* count,
                      cudaStream_t stream) {
  PageBook b;
  if (const int rc = check_book(book, true, &b); rc != TXL_OK) return rc;
  if (!pointers_ok(4, new_id, copy_src, copy_dst, count)) return TXL_ERR_INVALID_ARG;
  const BookRanges br = ranges(b);
  const Range outs[] = {range_of(new_id, ints(b.n_pages)), range_of(copy_src, ints(b.n_pages)),
                        range_of(copy_dst, ints(b.n_pages)), range_of(count, ints(1)), br.r[0], br.r[1], br.r[2],
                        br.r[3]};
  const Range none[] = {Range{0, 0}};
  if (aliased(outs, none)) return TXL_ERR_ALIAS;
  unsigned int* status;
  if (status_word(&status) != TXL_OK) return TXL_ERR_CUDA;
  return from_cuda(txl::launch_pages_compact(b, new_id, copy_src, copy_dst, count, status, stream));
}

size_t txl_relattn_paged_workspace_bytes(int n, int T, int H, int D, txl_dtype dtype) {
  if (n < 0 || T < 0 || H <= 0 || D <= 0 || !type_ok(dtype)) return 0;
  return txl::paged_workspace_bytes(n, T, H, D, dtype == TXL_BF16);
}

int txl_relattn_forward_paged(const void* q, const void* k_pages, const void* v_pages, const txl_page_book* book,
                              const int* slots, const int* cu, int n, int T, int max_new, const void* r,
                              const float* bias_u, const float* bias_v, void* o, float* lse, int H, int D, int n_r,
                              float scale, txl_dtype dtype, txl_dtype o_dtype, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  PageBook b;
  if (const int rc = check_book(book, false, &b); rc != TXL_OK) return rc;
  if (n < 0 || T < 0 || max_new < 0 || H <= 0 || D <= 0 || n_r < 0 || !type_ok(dtype) || !type_ok(o_dtype) ||
      !std::isfinite(scale))
    return TXL_ERR_INVALID_ARG;
  if (n == 0 || T == 0 || max_new == 0) return TXL_OK;
  if (max_new > T) max_new = T;
  const size_t es = size_of(dtype);
  if (!pointers_ok(dtype == TXL_BF16 ? 16 : 4, static_cast<const char*>(q), static_cast<const char*>(k_pages),
                   static_cast<const char*>(v_pages), static_cast<const char*>(r)) ||
      !pointers_ok(16, static_cast<const char*>(o)) || !pointers_ok(4, slots, cu) ||
      !pointers_ok(4, bias_u, bias_v) || !aligned(lse, 4) || n_r == 0)
    return TXL_ERR_INVALID_ARG;
  if (n > txl::kMaxSlots || H > 65535 || T > (1 << 30)) return TXL_ERR_UNSUPPORTED;
  if (dtype == TXL_F32 ? (o_dtype != TXL_F32 || D > 256) : (D != 64 && D != 128)) return TXL_ERR_UNSUPPORTED;
  if (!pointers_ok(256, static_cast<const char*>(workspace)) ||
      workspace_bytes < txl_relattn_paged_workspace_bytes(n, T, H, D, dtype))
    return TXL_ERR_INVALID_ARG;
  const size_t hd = static_cast<size_t>(H) * D;
  const size_t pool = static_cast<size_t>(b.n_pages) * hd * b.page_rows * es;
  const Range outs[] = {range_of(o, T * hd * size_of(o_dtype)), range_of(lse, static_cast<size_t>(H) * T * 4),
                        range_of(workspace, workspace_bytes)};
  const BookRanges br = ranges(b);
  const Range ins[] = {range_of(q, T * hd * es), range_of(k_pages, pool), range_of(v_pages, pool),
                       range_of(r, n_r * hd * es), range_of(bias_u, hd * 4), range_of(bias_v, hd * 4),
                       range_of(slots, ints(n)), range_of(cu, ints(n + 1LL)), br.r[0], br.r[1], br.r[2]};
  if (aliased(outs, ins)) return TXL_ERR_ALIAS;
  txl::PagedAttn a{b, q, k_pages, v_pages, r, bias_u, bias_v, o, lse, slots, cu, n, T, max_new, H, D, n_r, scale,
                   dtype == TXL_BF16, o_dtype == TXL_BF16, workspace};
  txl::WaitCtl wc;
  if (txl::api_wait_ctl(&wc) != TXL_OK) return TXL_ERR_CUDA;
  if (a.bf16) wc.inject_stall = txl::api_take_stall();
  return from_cuda(txl::launch_paged_attn(a, wc, stream));
}

int txl_debug_paged_pieces(int kind, int D, int H, int n, const int* start, const int* rows, const int* n_new,
                           int ctas, int* out, int cap) {
  if (kind < 0 || kind > 2 || (kind == 0 && D != 64 && D != 128) || H <= 0 || n < 0 || ctas <= 0 || ctas > 1023 || cap < 0 || start == nullptr ||
      rows == nullptr || n_new == nullptr || out == nullptr)
    return -2;
  for (int i = 0; i < n; ++i)
    if (start[i] < 0 || rows[i] < 0 || n_new[i] <= 0) return -2;
  return txl::paged_pieces(kind, D, H, n, start, rows, n_new, ctas, out, cap);
}

}  // extern "C"
