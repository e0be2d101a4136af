// Joins the pieces of the units that the division of the paged attention's
// work cut (paged_plan.cuh): with top = max_c lse_c over a unit's pieces c and
// w_c = 2^(lse_c - top),
//   o = sum_c w_c o_c / sum_c w_c,   lse = top + log2 sum_c w_c,
// the pieces taken in key order.
//
// A CTA has up to 16 rows of the unit whose first piece a CTA of the attention
// kernel had, if any.  Bound by latency: the pieces lie in L2, at most one unit
// per CTA of that kernel is cut, and most have few pieces.  So a thread takes
// its values of a row through all pieces with a running maximum and sum of its
// own, the loads of several pieces, and of their lse, in flight at once: behind
// the cut's own load one trip to L2, no barrier.  (Maxima, sums and rows in
// three passes over the pieces, with barriers between: 3.4 us of the 10.4 of a
// single token over 512 rows, 9.0 so.)  Units of tiles are nearly all cut in
// two: 2 pieces in flight and 16 rows a CTA, 1 us of 87 less for 22 sequences of
// 512 tokens over 512 rows than 4 and 32; fp32's have more, 21.7 us
// with 4 in flight against 22.9 (5 sequences of up to 130 tokens).
#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"
#include "pdl.cuh"
#include "txl_device.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int kThreads = 128, kRows = 16;

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

// One unit's rows r0 .. r0 + rows - 1: VECS values a thread and turn, AHEAD
// pieces in flight.
template <int VECS, int AHEAD, typename TO, typename V>
__device__ __forceinline__ void join_rows(const JoinPart& j, const PlanCut& cut, int first, int r0, int rows, TO* o,
                                          float* lse, int T, int H, int D) {
  constexpr int kWide = sizeof(V) / 4;
  const size_t size = static_cast<size_t>(plan_part(j.rows, D));
  const int cols = D / kWide, total = rows * cols, lse_at = j.rows * D + r0;
  for (int e0 = threadIdx.x; e0 < total; e0 += kThreads * VECS) {
    V acc[VECS];
    float top[VECS], sum[VECS];
    int row[VECS];
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      acc[v] = V{};
      top[v] = -INFINITY;
      sum[v] = 0.f;
      row[v] = min(e0 + v * kThreads, total - 1) / cols;
    }
    for (int c0 = 0; c0 < cut.pieces; c0 += AHEAD) {
      V val[AHEAD][VECS];
      float l[AHEAD][VECS];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int c = min(c0 + a, cut.pieces - 1);
        const float* from = j.part + plan_place(first + c, c) * size;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
          val[a][v] = reinterpret_cast<const V*>(from + r0 * D)[min(e0 + v * kThreads, total - 1)];
          l[a][v] = from[lse_at + row[v]];
        }
      }
#pragma unroll
      for (int v = 0; v < VECS; ++v) {
        float best = top[v];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) best = c0 + a < cut.pieces ? fmaxf(best, l[a][v]) : best;
        const float eff = best == -INFINITY ? 0.f : best;  // no visible key so far: every weight is 0
        const float keep = ex2(top[v] - eff);
        top[v] = best;
        acc[v] = times(acc[v], keep);
        sum[v] *= keep;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
          if (c0 + a < cut.pieces) {
            const float w = ex2(l[a][v] - eff);
            add(acc[v], w, val[a][v]);
            sum[v] += w;
          }
      }
    }
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      const int e = e0 + v * kThreads, col = e - row[v] * cols;
      if (e >= total) continue;
      const bool none = top[v] == -INFINITY;
      put(o + (static_cast<size_t>(cut.row0 + r0 + row[v]) * H + cut.h) * D + col * kWide,
          times(acc[v], none ? 0.f : 1.f / sum[v]));
      if (col == 0 && lse != nullptr)
        lse[static_cast<size_t>(cut.h) * T + cut.row0 + r0 + row[v]] =
            none ? -INFINITY : (top[v] + log2f(sum[v])) * 0.69314718055994531f;
    }
  }
}

// V: float, or float4 where D is a multiple of 4 (every row then starts on a
// 16-byte boundary).  DC: D where it is known, or 0.
template <typename TO, typename V, int DC>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const JoinPart x, const JoinPart y, TO* o, float* lse,
                                                              int T, int H, int d_arg) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int D = DC > 0 ? DC : d_arg;
  // Blocks of x first, each unit's blocks of 16 rows together.
  const int bx = (x.rows + kRows - 1) / kRows, by = (y.rows + kRows - 1) / kRows;
  const bool second = static_cast<int>(blockIdx.x) >= x.ctas * bx;
  const JoinPart& j = second ? y : x;
  const int b = static_cast<int>(blockIdx.x) - (second ? x.ctas * bx : 0), per = second ? by : bx;
  const int first = b / per, r0 = b % per * kRows;
  const PlanCut cut = j.cuts[first];
  if (cut.pieces == 0 || r0 >= cut.nq) return;
  const int rows = min(kRows, cut.nq - r0);
  if (rows <= kDecodeRows)  // up to 128 values a row of four
    join_rows<1, 8, TO, V>(j, cut, first, r0, rows, o, lse, T, H, D);
  else
    join_rows<2, (DC > 0 ? 2 : 4), TO, V>(j, cut, first, r0, rows, o, lse, T, H, D);
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
