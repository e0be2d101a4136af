// Joins the pieces of the units that the division of the paged attention's
// work cut (paged_plan.cuh): with top = max_c lse_c over a unit's pieces c and
// w_c = 2^(lse_c - top),
//   o = sum_c w_c o_c / sum_c w_c,   lse = top + log2 sum_c w_c,
// the pieces taken in key order.
//
// A CTA has up to 32 rows of the unit whose first piece CTA blockIdx.x of the
// attention kernel had, if any.  Bound by latency: the pieces lie in L2, and at
// most one unit per CTA of that kernel is cut.
#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"
#include "pdl.cuh"
#include "txl_device.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int kThreads = 128, kRows = 32, kVals = 8;

template <typename TO>
__device__ __forceinline__ void put(TO* p, float x);
template <>
__device__ __forceinline__ void put(float* p, float x) {
  *p = x;
}
template <>
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) {
  *p = __float2bfloat16(x);
}

template <typename TO>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const JoinPart x, const JoinPart y, TO* o, float* lse,
                                                              int T, int H, int D) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float s_top[kRows], s_inv[kRows];
  const bool second = static_cast<int>(blockIdx.x) >= x.ctas;
  const JoinPart& j = second ? y : x;
  const int first = static_cast<int>(blockIdx.x) - (second ? x.ctas : 0);
  const int r0 = blockIdx.y * kRows;
  if (r0 >= j.rows) return;
  const PlanCut cut = j.cuts[first];
  if (cut.pieces == 0 || r0 >= cut.nq) return;
  const int tid = threadIdx.x, rows = min(kRows, cut.nq - r0);
  const size_t size = static_cast<size_t>(plan_part(j.rows, D));
  auto piece = [&](int c) { return j.part + plan_place(first + c, c) * size; };
  const int lse_at = j.rows * D + r0;
  if (tid < rows) {
    float top = -INFINITY, sum = 0.f;
    for (int c = 0; c < cut.pieces; ++c) top = fmaxf(top, piece(c)[lse_at + tid]);
    const float eff = top == -INFINITY ? 0.f : top;
    for (int c = 0; c < cut.pieces; ++c) sum += ex2(piece(c)[lse_at + tid] - eff);
    s_top[tid] = eff;
    s_inv[tid] = top == -INFINITY ? 0.f : 1.f / sum;
    if (lse != nullptr)
      lse[static_cast<size_t>(cut.h) * T + cut.row0 + r0 + tid] =
          top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
  }
  __syncthreads();
  for (int e0 = 0; e0 < rows * D; e0 += kThreads * kVals) {
    float acc[kVals];
#pragma unroll
    for (int v = 0; v < kVals; ++v) acc[v] = 0.f;
    for (int c = 0; c < cut.pieces; ++c) {
      const float* from = piece(c);
#pragma unroll
      for (int v = 0; v < kVals; ++v) {
        const int e = e0 + v * kThreads + tid;
        if (e >= rows * D) continue;
        const int row = e / D;
        acc[v] = fmaf(ex2(from[lse_at + row] - s_top[row]), from[r0 * D + e], acc[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < kVals; ++v) {
      const int e = e0 + v * kThreads + tid;
      if (e >= rows * D) continue;
      const int row = e / D;
      put(o + (static_cast<size_t>(cut.row0 + r0 + row) * H + cut.h) * D + e % D, acc[v] * s_inv[row]);
    }
  }
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttn& a, const JoinPart& x, const JoinPart& y, cudaStream_t stream) {
  const int rows = x.rows > y.rows ? x.rows : y.rows;
  const dim3 grid(x.ctas + y.ctas, (rows + kRows - 1) / kRows);
  if (a.o_bf16)
    return launch_dependent(paged_join_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, x, y,
                            static_cast<__nv_bfloat16*>(a.o), a.lse, a.T, a.H, a.D);
  return launch_dependent(paged_join_kernel<float>, grid, dim3(kThreads), 0, stream, x, y, static_cast<float*>(a.o),
                          a.lse, a.T, a.H, a.D);
}

}  // namespace txl
