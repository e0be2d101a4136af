// Joins the pieces of the units that the division of the paged attention's
// work cut (paged_plan.cuh): with top = max_c lse_c over a unit's pieces c and
// w_c = 2^(lse_c - top),
//   o = sum_c w_c o_c / sum_c w_c,   lse = top + log2 sum_c w_c,
// the pieces taken in key order.
//
// A CTA has up to 32 rows of the unit whose first piece a CTA of the attention
// kernel had, if any.  Bound by latency: the pieces lie in L2, and at most one
// unit per CTA of that kernel is cut.  So the loads of several pieces are in
// flight at once: the weights are found by all threads (row by lane, pieces by
// warp), the rows by groups of four pieces.
#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"
#include "pdl.cuh"
#include "txl_device.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int kThreads = 128, kWarps = 4, kRows = 32, kAhead = 4, kVecs = 4;

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }
__device__ __forceinline__ void put(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}
__device__ __forceinline__ void add(float& a, float w, float x) { a = fmaf(w, x, a); }
__device__ __forceinline__ void add(float4& a, float w, float4 x) {
  a.x = fmaf(w, x.x, a.x);
  a.y = fmaf(w, x.y, a.y);
  a.z = fmaf(w, x.z, a.z);
  a.w = fmaf(w, x.w, a.w);
}
__device__ __forceinline__ float times(float a, float f) { return a * f; }
__device__ __forceinline__ float4 times(float4 a, float f) { return make_float4(a.x * f, a.y * f, a.z * f, a.w * f); }

// V: float, or float4 where D is a multiple of 4 (every row then starts on a
// 16-byte boundary).  DC: D where it is known, or 0.
template <typename TO, typename V, int DC>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const JoinPart x, const JoinPart y, TO* o, float* lse,
                                                              int T, int H, int d_arg) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float red[kWarps][kRows], s_top[kRows], s_inv[kRows];
  const int D = DC > 0 ? DC : d_arg;
  // Blocks of x first, each unit's blocks of 32 rows together.
  const int bx = (x.rows + kRows - 1) / kRows, by = (y.rows + kRows - 1) / kRows;
  const bool second = static_cast<int>(blockIdx.x) >= x.ctas * bx;
  const JoinPart& j = second ? y : x;
  const int b = static_cast<int>(blockIdx.x) - (second ? x.ctas * bx : 0), per = second ? by : bx;
  const int first = b / per, r0 = b % per * kRows;
  const PlanCut cut = j.cuts[first];
  if (cut.pieces == 0 || r0 >= cut.nq) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rows = min(kRows, cut.nq - r0);
  const size_t size = static_cast<size_t>(plan_part(j.rows, D));
  auto piece = [&](int c) { return j.part + plan_place(first + c, c) * size; };
  const int lse_at = j.rows * D + r0;

  const bool mine = lane < rows;
  float top = -INFINITY;
#pragma unroll 4
  for (int c = warp; c < cut.pieces; c += kWarps) top = fmaxf(top, mine ? piece(c)[lse_at + lane] : -INFINITY);
  red[warp][lane] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0][lane], red[1][lane]), fmaxf(red[2][lane], red[3][lane]));
  const float eff = top == -INFINITY ? 0.f : top;
  if (warp == 0) s_top[lane] = eff;
  __syncthreads();
  float sum = 0.f;
  if (warp == 0) {
#pragma unroll 4
    for (int c = 0; c < cut.pieces; ++c) sum += mine ? ex2(piece(c)[lse_at + lane] - eff) : 0.f;
    s_inv[lane] = top == -INFINITY ? 0.f : 1.f / sum;
    if (lse != nullptr && mine)
      lse[static_cast<size_t>(cut.h) * T + cut.row0 + r0 + lane] =
          top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
  }
  __syncthreads();

  constexpr int kWide = sizeof(V) / 4;
  const int cols = D / kWide, total = rows * cols;
  for (int e0 = 0; e0 < total; e0 += kThreads * kVecs) {
    V acc[kVecs];
    int row[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      acc[v] = V{};
      row[v] = min(e0 + v * kThreads + tid, total - 1) / cols;
    }
    for (int c0 = 0; c0 < cut.pieces; c0 += kAhead) {
      V val[kAhead][kVecs];
      float l[kAhead][kVecs];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const float* from = piece(min(c0 + a, cut.pieces - 1));
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          const int e = min(e0 + v * kThreads + tid, total - 1);
          val[a][v] = reinterpret_cast<const V*>(from + r0 * D)[e];
          l[a][v] = from[lse_at + row[v]];
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (c0 + a < cut.pieces) {
#pragma unroll
          for (int v = 0; v < kVecs; ++v) add(acc[v], ex2(l[a][v] - s_top[row[v]]), val[a][v]);
        }
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = e0 + v * kThreads + tid;
      if (e >= total) continue;
      put(o + (static_cast<size_t>(cut.row0 + r0 + row[v]) * H + cut.h) * D + (e - row[v] * cols) * kWide,
          times(acc[v], s_inv[row[v]]));
    }
  }
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttn& a, const JoinPart& x, const JoinPart& y, cudaStream_t stream) {
  auto blocks = [](const JoinPart& p) { return p.ctas * ((p.rows + kRows - 1) / kRows); };
  auto run = [&](auto kern, auto* o) {
    return launch_dependent(kern, dim3(blocks(x) + blocks(y)), dim3(kThreads), 0, stream, x, y, o, a.lse, a.T, a.H,
                            a.D);
  };
  if (a.o_bf16) {
    auto* o = static_cast<__nv_bfloat16*>(a.o);
    return a.D == 64 ? run(paged_join_kernel<__nv_bfloat16, float4, 64>, o)
                     : run(paged_join_kernel<__nv_bfloat16, float4, 128>, o);
  }
  auto* o = static_cast<float*>(a.o);
  if (a.bf16)
    return a.D == 64 ? run(paged_join_kernel<float, float4, 64>, o) : run(paged_join_kernel<float, float4, 128>, o);
  return a.D % 4 == 0 ? run(paged_join_kernel<float, float4, 0>, o) : run(paged_join_kernel<float, float, 0>, o);
}

}  // namespace txl
