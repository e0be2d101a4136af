// Internal interface of the paged memory (pages.cu, paged_attn.cu) to its C
// entry points (pages_api.cu).  Arguments are validated by the caller.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "txl_internal.h"

namespace txl {

// txl_page_book with the types the kernels use.
struct PageBook {
  int* table;
  int* start;
  int* rows;
  int* refs;
  int n_slots, max_pages, n_pages, page_rows;
};

constexpr int kMaxSlots = 16384;  // the reserve kernel keeps an int per slot and one per entry in shared memory

cudaError_t launch_pages_reserve(const PageBook& b, const int* slots, const int* cu, int n, int* granted,
                                 int* copy_src, int* copy_dst, unsigned int* status, cudaStream_t stream);
cudaError_t launch_pages_append(const PageBook& b, void* kp, void* vp, int H, int D, int elem, const int* slots,
                                const int* cu, int n, const int* granted, const int* copy_src, const int* copy_dst,
                                const void* kn, const void* vn, int T, unsigned int* status, cudaStream_t stream);
cudaError_t launch_pages_copy(void* kp, void* vp, int n_pages, long long page_bytes, const int* src, const int* dst,
                              int n, unsigned int* status, cudaStream_t stream);
cudaError_t launch_pages_fork(const PageBook& b, const int* src, const int* dst, int n, int* ok,
                              unsigned int* status, cudaStream_t stream);
cudaError_t launch_pages_free(const PageBook& b, const int* slots, const int* keep, int n, unsigned int* status,
                              cudaStream_t stream);
cudaError_t launch_pages_compact(const PageBook& b, int* new_id, int* copy_src, int* copy_dst, int* count,
                                 unsigned int* status, cudaStream_t stream);

// Attention of the new tokens of a ragged batch over their slots' rows.
struct PagedAttn {
  PageBook book;
  const void* q;  // [T, H, D]
  const void* kp;
  const void* vp;
  const void* r;  // [n_r, H, D]
  const float* bias_u;
  const float* bias_v;
  void* o;
  float* lse;  // [H, T] or nullptr
  const int* slots;
  const int* cu;
  int n, T, max_new, H, D, n_r;
  float scale;
  bool bf16, o_bf16;
  void* workspace;
};
size_t paged_workspace_bytes(int n, int T, int H, int D, bool bf16);
cudaError_t launch_paged_attn(const PagedAttn& a, const WaitCtl& wc, cudaStream_t stream);

// From api.cu: the status word with the wait bound, the test hook, the tensor-map encoder.
int api_wait_ctl(WaitCtl* wc);
int api_take_stall();  // the stall asked for by the test hook, once
PFN_cuTensorMapEncodeTiled_v12000 api_tensor_map_encoder();

}  // namespace txl
