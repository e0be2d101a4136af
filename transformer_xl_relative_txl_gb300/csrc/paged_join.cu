// Joins the pieces of the tile units that the division of the paged
// attention's work cut (paged_plan.cuh): with top = max_c lse_c over a unit's
// pieces c and w_c = 2^(lse_c - top),
//   o = sum_c w_c o_c / sum_c w_c,   lse = top + log2 sum_c w_c,
// the pieces taken in key order.
//
// CTA (c, y) has rows 32 y .. 32 y + 31 of the unit whose first piece CTA c of
// the tile kernel had, if any.  Bound by latency: the pieces lie in L2, and at
// most one unit per CTA of that kernel is cut (about 2 us behind it).
#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"
#include "pdl.cuh"
#include "txl_device.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int kThreads = 128, kRows = 32;

template <int D, bool O_BF16>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const TileCut* __restrict__ cuts,
                                                              const float* __restrict__ part, void* o, float* lse,
                                                              int T, int H) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float weight[kRows];
  const TileCut cut = cuts[blockIdx.x];
  const int r0 = blockIdx.y * kRows;
  if (cut.pieces == 0 || r0 >= cut.nq) return;
  const int tid = threadIdx.x, first = static_cast<int>(blockIdx.x);
  constexpr size_t kPart = tile_part(D);
  auto piece = [&](int c) { return part + plan_place(first + c, c) * kPart; };
  float top = -INFINITY, sum = 0.f;
  if (tid < kRows)
    for (int c = 0; c < cut.pieces; ++c) top = fmaxf(top, piece(c)[kTileQueries * D + r0 + tid]);
  const float eff = top == -INFINITY ? 0.f : top;
  constexpr int kVecs = kRows * D / 4 / kThreads;
  float4 acc[kVecs];
#pragma unroll
  for (int e = 0; e < kVecs; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < cut.pieces; ++c) {
    const float* from = piece(c);
    float4 x[kVecs];
#pragma unroll
    for (int e = 0; e < kVecs; ++e) x[e] = reinterpret_cast<const float4*>(from + r0 * D)[tid + e * kThreads];
    if (tid < kRows) {
      const float w = ex2(from[kTileQueries * D + r0 + tid] - eff);
      sum += w;
      weight[tid] = w;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kVecs; ++e) {
      const float w = weight[(tid + e * kThreads) / (D / 4)];
      acc[e].x = fmaf(w, x[e].x, acc[e].x);
      acc[e].y = fmaf(w, x[e].y, acc[e].y);
      acc[e].z = fmaf(w, x[e].z, acc[e].z);
      acc[e].w = fmaf(w, x[e].w, acc[e].w);
    }
    __syncthreads();
  }
  if (tid < kRows) {
    weight[tid] = top == -INFINITY ? 0.f : 1.f / sum;
    if (lse != nullptr && r0 + tid < cut.nq)
      lse[static_cast<size_t>(cut.h) * T + cut.row0 + r0 + tid] =
          top == -INFINITY ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kVecs; ++e) {
    const int row = (tid + e * kThreads) / (D / 4), d = (tid + e * kThreads) % (D / 4) * 4;
    if (r0 + row >= cut.nq) continue;
    const float inv = weight[row];
    const size_t at = (static_cast<size_t>(cut.row0 + r0 + row) * H + cut.h) * D + d;
    if (O_BF16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o) + at) =
          make_uint2(pack_bf16x2(acc[e].x * inv, acc[e].y * inv), pack_bf16x2(acc[e].z * inv, acc[e].w * inv));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(o) + at) =
          make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv);
  }
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttn& a, const PlanSpace& s, int sms, cudaStream_t stream) {
  const dim3 grid(sms, kTileQueries / kRows);
  auto run = [&](auto kern) {
    return launch_dependent(kern, grid, dim3(kThreads), 0, stream, static_cast<const TileCut*>(s.cuts),
                            static_cast<const float*>(s.part[1]), a.o, a.lse, a.T, a.H);
  };
  if (a.D == 64) return a.o_bf16 ? run(paged_join_kernel<64, true>) : run(paged_join_kernel<64, false>);
  return a.o_bf16 ? run(paged_join_kernel<128, true>) : run(paged_join_kernel<128, false>);
}

}  // namespace txl
