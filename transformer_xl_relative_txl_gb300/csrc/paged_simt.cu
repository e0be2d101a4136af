// fp32 relative attention of new tokens over a paged memory on the CUDA cores,
// any head dimension up to 256.
//
//   s[t,j] = scale * ((q_t + u) . k_j + (q_t + v) . r_{m+t-j}),  j <= m + t
//   o_t = softmax(s[t,.]) V,  m = rows - new tokens
//
// A unit is 16 queries of one (sequence, head), a key step 32 rows; the units'
// steps are divided evenly over 3 CTAs per SM (paged_plan.cuh), so that few
// long sequences fill the GPU too.  (Up to D = 116 three fit an SM; up to 184 two
// and beyond it one, which take the equal ranges in turn.)  The distances that a step needs are 47
// consecutive rows of r, d = m + t - j for 16 t and 32 j.
//
// Bound by shared-memory reads: per 4 dimensions a warp's 4 queries x 32 keys
// take 32 fused multiply-adds an element and 28 wavefronts of 16-byte reads
// (keys and r rows by lane, queries broadcast).  Rows in shared memory are
// padded to an odd number of 16-byte pieces, so that a quarter warp's reads of
// consecutive rows meet different banks.  The step's loads are coalesced rows,
// 16 in flight per lane, hidden behind the other CTAs of the SM.  A ragged
// batch of 5 sequences of up to 130 tokens over up to 700 rows (4 heads, D = 40)
// takes 22 us: few steps a CTA, each a chain of its rows' loads and three
// barriers; 9 us are the two launches, the division and the join.  8 of 256 tokens
// over 512 rows (8 heads) take 289 us at D = 64, 14 TFLOP/s, and 759 at D = 128, 11.
// One token each for 64 sequences over 300 to 4500 rows (16 heads of 64): 940 us
// where reading the rows takes 170, since a step computes 16 queries whatever
// there are.  (4 CTAs an SM
// leave 128 registers a thread, which spill: 4% slower.  A step's rows held in
// registers while the step before is computed: they spill, the same time.)
#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"
#include "pdl.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int kThreads = 128;
constexpr int BQ = kSimtQueries, BK = 32, BR = BQ + BK - 1;
constexpr int kPs = BQ + 2;  // floats of a key's row of weights

struct Unit {
  int h, row0, nq, t0, nks, d0, start, last, slot, index, pieces;  // nks 0: no more
};

struct Params {
  PlanArgs args;
  const float* q;
  const float* kp;
  const float* vp;
  const float* r;
  const float* bias_u;
  const float* bias_v;
  float* o;
  float* lse;
  int D, log_page;
  float scale_log2e;
  PlanCut* cuts;
  float* part;
};

constexpr int kRing = 64;  // units are found up to 32 at a time

struct Shared {
  PlanState plan;
  Unit unit[kRing];
};

__host__ __device__ constexpr int padded(int D) { return (D + 3) / 4 * 4; }
// Floats of a row in shared memory: an odd number of 16-byte pieces.
__host__ __device__ constexpr int stride_of(int D) { return padded(D) + (padded(D) / 4 % 2 == 0 ? 4 : 8); }

size_t smem_bytes(int D) {
  return (sizeof(Shared) + 15) / 16 * 16 +
         sizeof(float) * (2 * BQ * static_cast<size_t>(padded(D)) +
                          static_cast<size_t>(2 * BK + BR) * stride_of(D) + BK * kPs + 2 * BQ);
}

// NG: float4 columns of the output per thread (two rows each).
template <int NG>
__global__ void __launch_bounds__(kThreads, NG <= 2 ? kSimtPerSm : 1) paged_simt_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared* sh = reinterpret_cast<Shared*>(smem);
  const int D = p.D, DP = padded(D), S = stride_of(D), H = p.args.H;
  float* qu = reinterpret_cast<float*>(smem + (sizeof(Shared) + 15) / 16 * 16);  // [BQ][DP]
  float* qv = qu + BQ * DP;                                                      // [BQ][DP]
  float* ks = qv + BQ * DP;                                                      // [BK][S]
  float* vs = ks + BK * S;                                                       // [BK][S]
  float* rs = vs + BK * S;   // [BR][S], row x: distance d0 - x0 - (BK - 1) + x
  float* ps = rs + BR * S;   // [BK][kPs] weights by key
  float* al = ps + BK * kPs;  // [BQ] rescale of the row's accumulator
  float* li = al + BQ;        // [BQ] 1 / row sum
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  for (int e = tid; e < (2 * BQ) * DP + (2 * BK + BR) * S; e += kThreads) qu[e] = 0.f;  // the padding stays zero
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (tid == 0) p.cuts[blockIdx.x] = PlanCut{0, 0, 0, 0};
  plan_begin<SimtUnits>(p.args, static_cast<int>(gridDim.x), &sh->plan);

  bool bad = false;
  int known = 0;  // warp 0: units found
  bool ended = false;
  for (int un = -1;; ++un) {
    Unit w{};
    if (un >= 0) {
      w = sh->unit[un % kRing];
      if (w.nks == 0) break;
    }
    if (warp == 0 && known == un + 1 && !ended) {  // units un + 1 ..., and behind the last one an empty one
      PlanFound f{};
      const int found = plan_batch<SimtUnits>(p.args, &sh->plan, un < 0, &f, &ended);
      if (lane < found) {
        const int i0 = f.qt * BQ;
        const Unit u{f.h,       f.s.tok0 + i0,           min(BQ, f.s.n - i0), f.p.t0,    f.p.nks, f.s.start + f.s.rows - f.s.n + i0,
                     f.s.start, f.s.start + f.s.rows - 1, f.s.slot,            f.p.index, f.p.pieces};
        if (u.pieces > 1 && u.index == 0) p.cuts[blockIdx.x] = PlanCut{u.row0, u.nq, u.h, u.pieces};
        sh->unit[(known + lane) % kRing] = u;
      }
      known += found;
      if (ended && lane == 0) sh->unit[known % kRing] = Unit{};
    }
    if (un < 0) {
      __syncthreads();
      continue;
    }
    for (int y = warp; y < BQ; y += kThreads / 32)
      for (int d = lane; d < D; d += 32) {
        const float x = y < w.nq ? p.q[(static_cast<size_t>(w.row0 + y) * H + w.h) * D + d] : 0.f;
        qu[y * DP + d] = x + p.bias_u[w.h * D + d];
        qv[y * DP + d] = x + p.bias_v[w.h * D + d];
      }
    const int* table = p.args.book.table + static_cast<size_t>(w.slot) * p.args.book.max_pages;
    const size_t head = (static_cast<size_t>(w.h) << p.log_page) * D;
    const size_t page = (static_cast<size_t>(H) << p.log_page) * D;
    float acc[NG][2][4];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[g][y][e] = 0.f;
    // Queries 4 warp .. 4 warp + 3 keep their maximum and sum here.
    float mx[4], sum[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) mx[y] = -INFINITY, sum[y] = 0.f;
    const int end = min(w.last, w.d0 + w.nq - 1);  // last row any query sees

    // Pages have at least 16 rows, a power of two, and steps are counted from a
    // page's first: each half of a step lies in one page.
    auto page_of = [&](int t, int half) {  // of rows 16 half .. 16 half + 15 of step t
      const int x = t * BK + 16 * half;
      return x + 15 >= w.start && x <= end ? table[x >> p.log_page] : 0;
    };
    int ids[2] = {page_of(w.t0, 0), page_of(w.t0, 1)};

    for (int t = w.t0; t < w.t0 + w.nks; ++t) {
      const int x0 = t * BK;
      // Rows of keys and values: warp + 4 y.  Rows that no query sees are not
      // read: weight 0 times a leftover that is no number would not be 0.
      bool on[BK / 4];
      size_t off[BK / 4];
#pragma unroll
      for (int y = 0; y < BK / 4; ++y) {
        const int x = x0 + warp + 4 * y;
        int id = -1;
        if (x >= w.start && x <= end) {
          id = ids[y / (BK / 8)];
          if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.args.book.n_pages)) bad = true, id = -1;
        }
        on[y] = id >= 0;
        off[y] = static_cast<size_t>(max(id, 0)) * page + head +
                 static_cast<size_t>(x & ((1 << p.log_page) - 1)) * D;
      }
      if (t + 1 < w.t0 + w.nks) {  // on their way while this step runs
        ids[0] = page_of(t + 1, 0);
        ids[1] = page_of(t + 1, 1);
      }
      const int dist0 = w.d0 - x0 - (BK - 1);  // distance of row 0 of rs
      __syncthreads();                         // the step before has read the tiles
      // 64 dimensions at a time: a step of up to that many waits once.
      for (int d0 = lane; d0 < D; d0 += 64) {
        float kx[2][BK / 4], vx[2][BK / 4], rx[2][BR / 4 + 1];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int d = d0 + 32 * c;
          const bool in = d < D;
#pragma unroll
          for (int y = 0; y < BK / 4; ++y) {
            kx[c][y] = in && on[y] ? p.kp[off[y] + d] : 0.f;
            vx[c][y] = in && on[y] ? p.vp[off[y] + d] : 0.f;
          }
#pragma unroll
          for (int y = 0; y < BR / 4 + 1; ++y) {
            const int row = warp + 4 * y, dist = dist0 + row;
            rx[c][y] = in && row < BR && dist >= 0 && dist < p.args.n_r
                           ? __ldg(p.r + (static_cast<size_t>(dist) * H + w.h) * D + d)
                           : 0.f;
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int d = d0 + 32 * c;
          if (d >= D) continue;
#pragma unroll
          for (int y = 0; y < BK / 4; ++y) {
            ks[(warp + 4 * y) * S + d] = kx[c][y];
            vs[(warp + 4 * y) * S + d] = vx[c][y];
          }
#pragma unroll
          for (int y = 0; y < BR / 4 + 1; ++y)
            if (warp + 4 * y < BR) rs[(warp + 4 * y) * S + d] = rx[c][y];
        }
      }
      __syncthreads();
      float z[4] = {0.f, 0.f, 0.f, 0.f};
      for (int d = 0; d < DP; d += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(ks + lane * S + d);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float4 a = *reinterpret_cast<const float4*>(qu + (4 * warp + y) * DP + d);
          const float4 b = *reinterpret_cast<const float4*>(qv + (4 * warp + y) * DP + d);
          const float4 r4 = *reinterpret_cast<const float4*>(rs + (4 * warp + y - lane + BK - 1) * S + d);
          z[y] = fmaf(a.x, k4.x, z[y]);
          z[y] = fmaf(a.y, k4.y, z[y]);
          z[y] = fmaf(a.z, k4.z, z[y]);
          z[y] = fmaf(a.w, k4.w, z[y]);
          z[y] = fmaf(b.x, r4.x, z[y]);
          z[y] = fmaf(b.y, r4.y, z[y]);
          z[y] = fmaf(b.z, r4.z, z[y]);
          z[y] = fmaf(b.w, r4.w, z[y]);
        }
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int row = 4 * warp + y, x = x0 + lane;
        const float s = x >= w.start && x <= min(w.last, w.d0 + row) ? z[y] * p.scale_log2e : -INFINITY;
        float best = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
        const float top = fmaxf(mx[y], best);
        const float f = top == -INFINITY ? 0.f : exp2f(s - top);
        const float keep = mx[y] == -INFINITY ? 0.f : exp2f(mx[y] - top);
        float part = f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        sum[y] = sum[y] * keep + part;
        mx[y] = top;
        ps[lane * kPs + row] = f;
        if (lane == 0) al[row] = keep;
      }
      __syncthreads();
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int e = tid + g * kThreads, rp = e & 7, c = e >> 3;  // rows 2 rp, 2 rp + 1, columns 4 c .. 4 c + 3
        if (4 * c >= DP) continue;
        const float2 k2 = *reinterpret_cast<const float2*>(al + 2 * rp);
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[g][0][x] *= k2.x, acc[g][1][x] *= k2.y;
#pragma unroll 8
        for (int j = 0; j < BK; ++j) {
          const float2 f = *reinterpret_cast<const float2*>(ps + j * kPs + 2 * rp);
          const float4 v4 = *reinterpret_cast<const float4*>(vs + j * S + 4 * c);
          acc[g][0][0] = fmaf(f.x, v4.x, acc[g][0][0]);
          acc[g][0][1] = fmaf(f.x, v4.y, acc[g][0][1]);
          acc[g][0][2] = fmaf(f.x, v4.z, acc[g][0][2]);
          acc[g][0][3] = fmaf(f.x, v4.w, acc[g][0][3]);
          acc[g][1][0] = fmaf(f.y, v4.x, acc[g][1][0]);
          acc[g][1][1] = fmaf(f.y, v4.y, acc[g][1][1]);
          acc[g][1][2] = fmaf(f.y, v4.z, acc[g][1][2]);
          acc[g][1][3] = fmaf(f.y, v4.w, acc[g][1][3]);
        }
      }
    }

    const bool whole = w.pieces == 1;
    float* out = p.part + plan_place(static_cast<int>(blockIdx.x), w.index) * plan_part(BQ, D);
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (lane == 0) {
        const int row = 4 * warp + y;
        const bool none = mx[y] == -INFINITY;
        const float lse2 = none ? -INFINITY : mx[y] + log2f(sum[y]);
        li[row] = none ? 0.f : 1.f / sum[y];
        if (!whole)
          out[BQ * D + row] = lse2;
        else if (p.lse != nullptr && row < w.nq)
          p.lse[static_cast<size_t>(w.h) * p.args.T + w.row0 + row] = none ? -INFINITY : lse2 * 0.69314718055994531f;
      }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int e = tid + g * kThreads, rp = e & 7, c = e >> 3;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int row = 2 * rp + y;
        if (row >= w.nq) continue;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int d = 4 * c + x;
          if (d >= D) continue;
          const float f = acc[g][y][x] * li[row];
          if (whole)
            p.o[(static_cast<size_t>(w.row0 + row) * H + w.h) * D + d] = f;
          else
            out[row * D + d] = f;
        }
      }
    }
    __syncthreads();  // the next unit is there; this one's shared rows are free
  }
  if (bad) atomicOr(p.args.status, kStatusPagesBit);
}

template <int NG>
cudaError_t launch(const Params& p, int sms, cudaStream_t stream) {
  const size_t smem = smem_bytes(p.D);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<NG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem_bytes(256)));
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(paged_simt_kernel<NG>, dim3(kSimtPerSm * sms), dim3(kThreads), smem, stream, p);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedAttn& a, const PlanSpace& s, int sms, unsigned int* status,
                              cudaStream_t stream) {
  const Params p{plan_args(a, status),
                 static_cast<const float*>(a.q),
                 static_cast<const float*>(a.kp),
                 static_cast<const float*>(a.vp),
                 static_cast<const float*>(a.r),
                 a.bias_u,
                 a.bias_v,
                 static_cast<float*>(a.o),
                 a.lse,
                 a.D,
                 __builtin_ctz(a.book.page_rows),
                 a.scale * 1.4426950408889634f,
                 s.simt.cuts,
                 s.simt.part};
  if (a.D <= 64) return launch<1>(p, sms, stream);
  if (a.D <= 128) return launch<2>(p, sms, stream);
  return launch<4>(p, sms, stream);
}

}  // namespace txl
