// Relative attention of new tokens over a paged memory on the CUDA cores,
// any head dimension up to 256, fp32 arithmetic.
//
//   s[t,j] = scale * ((q_t + u) . k_j + (q_t + v) . r_{m+t-j}),  j <= m + t
//   o_t = softmax(s[t,.]) V,  m = rows - new tokens
//
// A CTA takes 16 queries of one (sequence, head) and walks the keys in tiles
// of 32 with a running maximum and sum per row.  The distances a tile needs
// are 47 consecutive rows of r, d = m + t - j for 16 t and 32 j.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>

#include "pages.h"
#include "pdl.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int kThreads = 128;
constexpr int BQ = 16, BK = 32, BR = BQ + BK - 1;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

size_t smem_bytes(int D) {
  return sizeof(float) * (static_cast<size_t>(2 * BQ) * D + static_cast<size_t>(2 * BK + BR) * (D + 1) +
                          BQ * (BK + 1) + 2 * BQ);
}

template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(const PagedAttn a, unsigned int* status) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  extern __shared__ float sm[];
  const int D = a.D, H = a.H, S = D + 1;
  float* qu = sm;                  // [BQ][D]
  float* qv = qu + BQ * D;         // [BQ][D]
  float* ks = qv + BQ * D;         // [BK][S]
  float* vs = ks + BK * S;         // [BK][S]
  float* rs = vs + BK * S;         // [BR][S], row x: distance d0 + x
  float* ps = rs + BR * S;         // [BQ][BK + 1] weights
  float* al = ps + BQ * (BK + 1);  // [BQ] rescale of the row's accumulator
  float* li = al + BQ;             // [BQ] 1 / row sum

  const int i = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const PageBook& b = a.book;
  const int t0 = a.cu[i], n = a.cu[i + 1] - t0, q0 = blockIdx.x * BQ;
  const int s = a.slots[i];
  bool ok = s >= 0 && s < b.n_slots && n >= 0 && n <= a.max_new && t0 >= 0 && static_cast<long long>(t0) + n <= a.T;
  int start = 0, rows = 0;
  if (ok) {
    start = b.start[s];
    rows = b.rows[s];
    ok = start >= 0 && start < b.page_rows && rows >= 0 && rows <= a.n_r &&
         static_cast<long long>(start) + rows <= static_cast<long long>(b.max_pages) * b.page_rows;
  }
  if (!ok) {
    if (tid == 0) atomicOr(status, kStatusPagesBit);
    return;
  }
  if (q0 >= n) return;
  const int m = rows - n;  // position of query 0; negative: queries before row 0 see nothing
  const int nq = min(BQ, n - q0);
  const T* q = static_cast<const T*>(a.q);
  const T* r = static_cast<const T*>(a.r);
  for (int e = tid; e < BQ * D; e += kThreads) {
    const int y = e / D, d = e % D;
    const float x = y < nq ? to_f(q[(static_cast<size_t>(t0 + q0 + y) * H + h) * D + d]) : 0.f;
    qu[e] = x + a.bias_u[h * D + d];
    qv[e] = x + a.bias_v[h * D + d];
  }
  const int* table = b.table + static_cast<size_t>(s) * b.max_pages;
  const size_t page = static_cast<size_t>(H) * b.page_rows * D;
  float acc[2][BQ];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int y = 0; y < BQ; ++y) acc[c][y] = 0.f;
  // Rows 4 warp .. 4 warp + 3 of the tile keep their maximum and sum here.
  float mx[4], sum[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) mx[y] = -INFINITY, sum[y] = 0.f;

  const int last = min(rows - 1, m + q0 + nq - 1);  // last key any row sees
  bool bad = false;
  for (int j0 = 0; j0 <= last; j0 += BK) {
    __syncthreads();
    for (int e = tid; e < BK * D; e += kThreads) {
      const int y = e / D, d = e % D, j = j0 + y;
      float kx = 0.f, vx = 0.f;  // rows past the last are not read: weight 0 times a leftover could be NaN
      if (j <= last) {
        const int x = start + j, id = table[x / b.page_rows];
        if (id >= 0 && id < b.n_pages) {
          const size_t at = id * page + (static_cast<size_t>(h) * b.page_rows + x % b.page_rows) * D + d;
          kx = to_f(static_cast<const T*>(a.kp)[at]);
          vx = to_f(static_cast<const T*>(a.vp)[at]);
        } else {
          bad = true;
        }
      }
      ks[y * S + d] = kx;
      vs[y * S + d] = vx;
    }
    const int d0 = m + q0 - j0 - (BK - 1);  // distance of row 0 of rs
    for (int e = tid; e < BR * D; e += kThreads) {
      const int y = e / D, d = e % D, dist = d0 + y;
      rs[y * S + d] = dist >= 0 && dist < a.n_r ? to_f(r[(static_cast<size_t>(dist) * H + h) * D + d]) : 0.f;
    }
    __syncthreads();
    float z[4] = {0.f, 0.f, 0.f, 0.f};
    for (int d = 0; d < D; ++d) {
      const float kx = ks[lane * S + d];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int row = 4 * warp + y;
        z[y] = fmaf(qu[row * D + d], kx, z[y]);
        z[y] = fmaf(qv[row * D + d], rs[(row - lane + BK - 1) * S + d], z[y]);
      }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int row = 4 * warp + y, j = j0 + lane;
      const float x = j <= last && j <= m + q0 + row ? z[y] * a.scale : -INFINITY;
      float best = x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
      const float top = fmaxf(mx[y], best);
      const float w = top == -INFINITY ? 0.f : expf(x - top);
      const float scale_old = mx[y] == -INFINITY ? 0.f : expf(mx[y] - top);
      float part = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      sum[y] = sum[y] * scale_old + part;
      mx[y] = top;
      ps[row * (BK + 1) + lane] = w;
      if (lane == 0) al[row] = scale_old;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int d = tid + c * kThreads;
      if (d >= D) continue;
#pragma unroll
      for (int y = 0; y < BQ; ++y) acc[c][y] *= al[y];
      for (int j = 0; j < BK; ++j) {
        const float x = vs[j * S + d];
#pragma unroll
        for (int y = 0; y < BQ; ++y) acc[c][y] = fmaf(ps[y * (BK + 1) + j], x, acc[c][y]);
      }
    }
  }
  if (bad) atomicOr(status, kStatusPagesBit);
#pragma unroll
  for (int y = 0; y < 4; ++y)
    if (lane == 0) {
      const int row = 4 * warp + y;
      li[row] = mx[y] == -INFINITY ? 0.f : 1.f / sum[y];
      if (a.lse != nullptr && row < nq)
        a.lse[static_cast<size_t>(h) * a.T + t0 + q0 + row] = mx[y] == -INFINITY ? -INFINITY : mx[y] + logf(sum[y]);
    }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int d = tid + c * kThreads;
    if (d >= D) continue;
#pragma unroll
    for (int y = 0; y < BQ; ++y)
      if (y < nq)
        put(static_cast<TO*>(a.o) + (static_cast<size_t>(t0 + q0 + y) * H + h) * D + d, acc[c][y] * li[y]);
  }
}

template <typename T, typename TO>
cudaError_t launch(const PagedAttn& a, unsigned int* status, cudaStream_t stream) {
  const size_t smem = smem_bytes(a.D);
  const cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<T, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const dim3 grid((a.max_new + BQ - 1) / BQ, a.H, a.n);
  return launch_dependent(paged_simt_kernel<T, TO>, grid, dim3(kThreads), smem, stream, a, status);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedAttn& a, unsigned int* status, cudaStream_t stream) {
  if (!a.bf16) return launch<float, float>(a, status, stream);
  return a.o_bf16 ? launch<__nv_bfloat16, __nv_bfloat16>(a, status, stream)
                  : launch<__nv_bfloat16, float>(a, status, stream);
}

}  // namespace txl
