// Relative attention of a few new tokens per sequence (up to 4) over a paged
// memory, bf16 storage, head dimension 64 or 128.
//
//   s[t,j] = scale * ((q_t + u) . k_j + (q_t + v) . r_{m+t-j}),  j <= m + t
//
// Bound by reading K and V once: 2 * 2 D bytes per (sequence, head, row), and
// about 6 D flops per query on them, far below what a tensor core tile of 128
// queries would need to pay.  So the kernel's care is the loads: a producer
// warp keeps NS key tiles of K, V and r in flight per CTA by TMA (two CTAs per
// SM), straight from the pages, and as many warps consume whole tiles in turn,
// each with a softmax state of its own; they meet only at the end of a unit.
//
// The products run as mma.sync m16n8k16 with the long operand on the M side:
// S^T[keys x 8] = K [keys x D] Q^T, O^T[D x 8] += V^T P.  The 8 columns hold
// 4 queries as two bf16 parts each, x = hi + lo: (q + u) and (q + v), scaled
// in fp32, and the weights keep 16 bits of significand that way, at no cost,
// since the columns are there.  Adding the two columns of a query is an add
// of two accumulators of one thread.
//
// The distance term needs no shift in registers: key c of a tile meets row
// BK-1-c + t of the tile of r that starts at distance m - j0 - (BK-1), so
// query t's rows of r are addressed upside down by ldmatrix, and the product
// accumulates on top of the content term; the other queries' columns of the
// right-hand side are zero for it.
//
// Measured: 64 sequences of one token over 300 to 4500 rows (16 heads of 64,
// 757 MB) 126 us, 6.0 TB/s, 89% of a copy's rate; 48 over 1600 to 8100 rows (8
// heads of 128, pages of 32 rows, 1.02 GB) 175 us, 5.8 TB/s, 86%.  What is left
// is the CTAs' head and tail, about 8 us, and the join behind them.  One token
// over 512 rows (8 heads of 64): 9 us, of which the launches and waits take 2,
// the division 2, the tiles 3, the join 2.
#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"
#include "pdl.cuh"
#include "relattn_tc_common.cuh"
#include "txl_device.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

template <int D>
struct Cfg {
  static constexpr int BK = D == 64 ? 64 : 32;  // rows of a key tile: 8 KB either way
  // Stages, and consumer warps.  Tile g lies in stage g % NS and goes to warp
  // g % kWarps.  With as many of one as of the other a stage is one warp's for
  // good, which then sees every phase of the stage's barriers; a warp that
  // met only some of them could take an old phase of equal parity for the one
  // it waits for.
  static constexpr int NS = D == 64 ? 4 : 3;
  static constexpr int kWarps = NS;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int BR = BK + 8;  // rows of r: 3 more than a tile for the later queries
  static constexpr int kBoxes = D / 64;
  static constexpr int kTile = BK * D * 2, kTileR = BR * D * 2;
  static constexpr int kStage = 2 * kTile + kTileR;
  static constexpr int kRow = D + 2;  // a query's partial result: o, m, l
  static constexpr int kOffPart = NS * kStage;
  static constexpr int kQuery = kDecodeRows * D * 2 + 2 * D * 4;  // a unit's rows of q, u and v
  static constexpr int kOffQ = kOffPart + 2 * kWarps * kDecodeRows * kRow * 4;
  static constexpr int kOffBar = kOffQ + 2 * kQuery;
  static constexpr int kBarBytes = 1792;
  static constexpr int kSmem = kOffBar + kBarBytes + 1024;
  using Units = PlanUnits<DecodeCost, BK, 0, 1, kDecodeRows>;  // DecodeUnits64, DecodeUnits32
};

struct Params {
  PlanArgs args;
  const __nv_bfloat16* q;
  const float* bias_u;
  const float* bias_v;
  void* o;
  float* lse;
  float scale_log2e;
  PlanCut* cuts;
  float* part;
  unsigned long long wait_ns;
  bool ahead_of_tiles;
  int inject_stall;  // test hook: the producer (even CTAs) or a consumer (odd ones) stops behind a unit's first tile
};

// A unit as the producer publishes it; nks 0: the CTA has no more.
struct Unit {
  int h, tok0, n, start, last, t0, nks, index, pieces;
};

struct Bars {
  uint64_t full[4], empty[4], joined;
  uint64_t q_full[2], q_empty[2];  // by unit parity: the unit and its queries are there; read
  Unit unit[2];
  PlanState plan;
  int abort;
};

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Four bytes to shared memory, and an arrival on `bar` once this thread's
// copies so far have landed.
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The bf16 part `lo` (0: the value rounded, 1: what the rounding left) of a
// and b, packed.
__device__ __forceinline__ uint32_t split_part(float a, float b, bool lo) {
  const uint32_t hi = pack_bf16x2(a, b);
  return lo ? pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi)) : hi;
}

template <int D, bool O_BF16>
__global__ void __launch_bounds__(Cfg<D>::kThreads, kDecodePerSm)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_r, const Params p) {
  using C = Cfg<D>;
  constexpr int BK = C::BK, NS = C::NS, kWarps = C::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* joint = reinterpret_cast<float*>(smem + C::kOffPart);
  uint8_t* queries = smem + C::kOffQ;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  static_assert(sizeof(Bars) <= C::kBarBytes, "barrier block too large");
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->joined, kWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->q_full[s], 33);  // the lanes' copies, and the unit
      mbar_init(&bars->q_empty[s], kWarps);
    }
    bars->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (threadIdx.x == 0) p.cuts[blockIdx.x] = PlanCut{0, 0, 0, 0};
  if (p.ahead_of_tiles) {  // most batches of longer entries have none of these
    bool any = false;
    for (int i = threadIdx.x; i < p.args.n; i += blockDim.x) {
      const int n = p.args.cu[i + 1] - p.args.cu[i];
      any |= n >= 1 && n <= kDecodeRows;
    }
    if (!__syncthreads_or(any)) return;
  }
  plan_begin<typename C::Units>(p.args, static_cast<int>(gridDim.x), &bars->plan);
  const uint64_t wait_ns = p.wait_ns;

  if (warp == kWarps) {
    // ============================== producer ===============================
    PlanFound w{};  // the unit at hand, of every lane
    auto of_lane = [](const PlanFound& f, int x) {
      PlanFound g;
      g.s.tok0 = __shfl_sync(0xffffffffu, f.s.tok0, x);
      g.s.n = __shfl_sync(0xffffffffu, f.s.n, x);
      g.s.slot = __shfl_sync(0xffffffffu, f.s.slot, x);
      g.s.start = __shfl_sync(0xffffffffu, f.s.start, x);
      g.s.rows = __shfl_sync(0xffffffffu, f.s.rows, x);
      g.h = __shfl_sync(0xffffffffu, f.h, x);
      g.p.t0 = __shfl_sync(0xffffffffu, f.p.t0, x);
      g.p.nks = __shfl_sync(0xffffffffu, f.p.nks, x);
      g.p.index = __shfl_sync(0xffffffffu, f.p.index, x);
      g.p.pieces = __shfl_sync(0xffffffffu, f.p.pieces, x);
      return g;
    };
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_r);
    }
    const int P = p.args.book.page_rows;
    const int box = min(P, BK), boxes = BK / box;  // a tile is `boxes` boxes of rows
    uint32_t g = 0, units = 0;
    bool ok = true, bad = false, stop = false;
    // The next unit and its queries, on their way while its tiles are loaded:
    // read by the consumers at the head of the unit, a global load's latency a
    // unit made 163 us of what then took 125 (64 sequences, see above).
    auto publish = [&](int nks) {
      const int s = units & 1;
      ok = warp_wait(&bars->q_empty[s], ((units >> 1) & 1) ^ 1, wait_ns, abort);
      if (!ok) return;
      if (nks > 0) {
        uint8_t* at = queries + s * C::kQuery;
        const int total = w.s.n * (D / 2);  // words of the queries' rows
        for (int e = lane; e < total; e += 32)
          copy4(at + e * 4, p.q + (static_cast<size_t>(w.s.tok0 + e / (D / 2)) * p.args.H + w.h) * D + e % (D / 2) * 2);
#pragma unroll
        for (int e = lane; e < D; e += 32) {
          copy4(at + kDecodeRows * D * 2 + e * 4, p.bias_u + w.h * D + e);
          copy4(at + kDecodeRows * D * 2 + (D + e) * 4, p.bias_v + w.h * D + e);
        }
      }
      copies_arrive(&bars->q_full[s]);
      if (lane == 0) {
        Unit u{};
        if (nks > 0)
          u = Unit{w.h, w.s.tok0, w.s.n, w.s.start, w.s.start + w.s.rows - 1, w.p.t0, nks, w.p.index, w.p.pieces};
        bars->unit[s] = u;
        if (u.pieces > 1 && u.index == 0) p.cuts[blockIdx.x] = PlanCut{u.tok0, u.n, u.h, u.pieces};
        mbar_arrive(&bars->q_full[s]);
      }
      ++units;
    };
    PlanFound batch{};
    int at = 0, found = 0;
    bool last_batch = false, first = true;
    for (;;) {
      if (at == found) {
        if (last_batch) break;
        found = plan_batch<typename C::Units>(p.args, &bars->plan, first, &batch, &last_batch);
        first = false;
        at = 0;
        if (found == 0) break;
      }
      w = of_lane(batch, at++);
      publish(w.p.nks);
      if (!ok) break;
      const int* row = p.args.book.table + static_cast<size_t>(w.s.slot) * p.args.book.max_pages;
      const int last = w.s.start + w.s.rows - 1;
      const int m = w.s.start + w.s.rows - w.s.n;
      int id = -1, id0 = -32;  // this lane's page of the boxes from id0 on
      for (int t = w.p.t0; t < w.p.t0 + w.p.nks; ++t, ++g) {
        if (p.inject_stall && t > w.p.t0 && blockIdx.x % 2 == 0) {
          stop = true;
          break;
        }
        if (t * boxes - id0 + boxes > 32) {  // the next 32 boxes' pages at once (boxes divides 32)
          id0 = t * boxes;
          const long long x = static_cast<long long>(id0 + lane) * box;
          id = -1;
          if (x <= last && x + box > w.s.start) {
            id = row[x / P];
            if (id < 0 || id >= p.args.book.n_pages) bad = true, id = p.args.book.n_pages;  // zero rows, nothing read
          }
        }
        const int s = g % NS;
        ok = warp_wait(&bars->empty[s], ((g / NS) & 1) ^ 1, wait_ns, abort);
        if (!ok) break;
        uint8_t* stage = smem + s * C::kStage;
        const uint32_t mask = __ballot_sync(0xffffffffu, id >= 0) >> (t * boxes - id0) & ((1u << boxes) - 1);
        if (lane == 0)
          mbar_arrive_expect_tx(&bars->full[s], C::kTileR + 2 * static_cast<uint32_t>(__popc(mask)) * box * D * 2);
        for (int y = 0; y < boxes; ++y) {
          const int page = __shfl_sync(0xffffffffu, id, t * boxes - id0 + y);
          if (lane != 0 || page < 0) continue;
          const int x = (t * BK + y * box) % P;
#pragma unroll
          for (int c = 0; c < C::kBoxes; ++c) {
            uint8_t* at = stage + c * BK * 128 + y * box * 128;
            tma_load_4d(at, &tm_k, &bars->full[s], c * 64, x, w.h, page);
            tma_load_4d(at + C::kTile, &tm_v, &bars->full[s], c * 64, x, w.h, page);
          }
        }
        if (lane == 0) {
#pragma unroll
          for (int c = 0; c < C::kBoxes; ++c)
            tma_load_3d(stage + 2 * C::kTile + c * C::BR * 128, &tm_r, &bars->full[s], c * 64, w.h,
                        m - t * BK - (BK - 1));
        }
        __syncwarp();
      }
      // (Another unit's tiles would be taken, by their number, for the rest of
      // this one's.)
      if (!ok || stop) break;
    }
    if (ok && !stop) publish(0);
    if (bad) atomicOr(p.args.status, kStatusPagesBit);
    if (!ok && lane == 0) report_timeout(abort, p.args.status);
    asm volatile("cp.async.wait_all;" ::: "memory");
    // This warp's copies land before the CTA may exit.
    for (uint32_t s = 0; s < NS && s < g; ++s) {
      const uint32_t n = s + ((g - 1 - s) / NS) * NS;
      mbar_wait_own(&bars->full[s], (n / NS) & 1, wait_ns);
    }
    return;
  }

  // =============================== consumers ================================
  const int col_q = lane >> 3, part = lane >> 2 & 1;  // query and part of this lane's right-hand column
  const int my_q = lane & 3;                          // query of this lane's accumulators
  uint32_t g = 0;
  bool ok = true;
  for (uint32_t units = 0;; ++units) {
    ok = warp_wait(&bars->q_full[units & 1], (units >> 1) & 1, wait_ns, abort);
    if (!ok) break;
    const Unit w = bars->unit[units & 1];
    const int n = w.n, h = w.h;
    // (q + u), (q + v) in log2 units, as right-hand fragments.
    uint32_t qu[D / 8], qv[D / 8];
    if (w.nks > 0) {
      const uint8_t* at = queries + (units & 1) * C::kQuery;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(at) + min(col_q, n - 1) * (D / 2);
      const float* bias = reinterpret_cast<const float*>(at + kDecodeRows * D * 2);
#pragma unroll
      for (int e = 0; e < D / 8; ++e) {
        const int d = e * 8 + 2 * (lane & 3);
        const uint32_t x = q[d / 2];
        const float f = p.scale_log2e, x0 = bf16_lo(x), x1 = bf16_hi(x);
        const float2 bu = *reinterpret_cast<const float2*>(bias + d);
        const float2 bv = *reinterpret_cast<const float2*>(bias + D + d);
        qu[e] = col_q < n ? split_part((x0 + bu.x) * f, (x1 + bu.y) * f, part) : 0u;
        qv[e] = col_q < n ? split_part((x0 + bv.x) * f, (x1 + bv.y) * f, part) : 0u;
      }
    }
    warp_arrive(&bars->q_empty[units & 1]);
    if (w.nks == 0) break;
    const int last = w.last;
    const int lim = last + 1 - n + my_q;  // last row this lane's query sees
    float m_run = -INFINITY, l_run = 0.f;
    float acc[D / 16][4];
#pragma unroll
    for (int e = 0; e < D / 16; ++e)
#pragma unroll
      for (int y = 0; y < 4; ++y) acc[e][y] = 0.f;

    // This warp's tiles: those that the CTA loaded as number g with
    // g % kWarps == warp.
    const uint32_t g0 = g;
    g += w.nks;
    for (uint32_t x = g0 + (warp + kWarps - g0 % kWarps) % kWarps; x < g; x += kWarps) {
      if (p.inject_stall && x > g0 && warp == 0 && blockIdx.x % 2 != 0) return;
      const int row0 = (w.t0 + static_cast<int>(x - g0)) * BK;
      const int s = x % NS;
      ok = warp_wait(&bars->full[s], (x / NS) & 1, wait_ns, abort);
      if (!ok) break;
      const uint32_t sk = smem_u32(smem + s * C::kStage), sv = sk + C::kTile, sr = sk + 2 * C::kTile;
      const int r16 = lane & 15, half = lane >> 4;
      float z[BK / 16][4];
#pragma unroll
      for (int y = 0; y < BK / 16; ++y) {
        z[y][0] = z[y][1] = z[y][2] = z[y][3] = 0.f;
        const int rk = 16 * y + r16;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          uint32_t a[4];
          ldsm4(sk + (e / 4) * BK * 128 + rk * 128 + ((((e % 4) * 2 + half) ^ (rk & 7)) << 4), a);
          mma16816(z[y], a, qu[2 * e], qu[2 * e + 1]);
        }
      }
      for (int t = 0; t < n; ++t) {
        const bool mine = col_q == t;
#pragma unroll
        for (int y = 0; y < BK / 16; ++y) {
          const int rr = BK - 1 - (16 * y + r16) + t;
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            uint32_t a[4];
            ldsm4(sr + (e / 4) * C::BR * 128 + rr * 128 + ((((e % 4) * 2 + half) ^ (rr & 7)) << 4), a);
            mma16816(z[y], a, mine ? qv[2 * e] : 0u, mine ? qv[2 * e + 1] : 0u);
          }
        }
      }
      // Scores of query my_q: rows row0 + 16 y + lane / 4 (+ 8).
      const bool edge = row0 < w.start || row0 + BK - 1 > last - (n - 1);
      float sc[BK / 16][2];
      float best = -INFINITY;
#pragma unroll
      for (int y = 0; y < BK / 16; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float f = z[y][2 * u] + z[y][2 * u + 1];
          if (edge) {
            const int row = row0 + 16 * y + 8 * u + (lane >> 2);
            f = row >= w.start && row <= lim ? f : -INFINITY;
          }
          sc[y][u] = f;
          best = fmaxf(best, f);
        }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
      const float m_new = fmaxf(m_run, best);
      const float m_eff = m_new == -INFINITY ? 0.f : m_new;
      if (__any_sync(0xffffffffu, m_new > m_run)) {
        const float f = ex2(m_run - m_eff);  // 2^-inf = 0 before the first visible row
        l_run *= f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[e][y] *= f;
        m_run = m_new;
      }
      uint32_t pt[BK / 16][2];  // weights as right-hand fragments
#pragma unroll
      for (int y = 0; y < BK / 16; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float f = ex2(sc[y][u] - m_eff);
          l_run += f;
          const float hi = __bfloat162float(__float2bfloat16(f));
          pt[y][u] = transpose8x8(pack_bf16x2(hi, f - hi));
        }
#pragma unroll
      for (int y = 0; y < BK / 16; ++y) {
        // Rows outside [start, last] hold leftovers: their values leave the
        // product as zeros, since 0 times NaN is not 0.
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (edge) {
          auto live = [&](int row) { return row >= w.start && row <= last; };
          const int row = row0 + 16 * y + 2 * (lane & 3);
          keep0 = (live(row) ? 0xffffu : 0u) | (live(row + 1) ? 0xffff0000u : 0u);
          keep1 = (live(row + 8) ? 0xffffu : 0u) | (live(row + 9) ? 0xffff0000u : 0u);
        }
        const int rv = 16 * y + (half << 3) + (lane & 7);
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          uint32_t a[4];
          ldsm4_t(sv + (e / 4) * BK * 128 + rv * 128 + ((((e % 4) * 2 + (lane >> 3 & 1)) ^ (rv & 7)) << 4), a);
          a[0] &= keep0, a[1] &= keep0, a[2] &= keep1, a[3] &= keep1;
          mma16816(acc[e], a, pt[y][0], pt[y][1]);
        }
      }
      warp_arrive(&bars->empty[s]);
    }
    if (!ok) break;

    // The warps' results meet; each warp joins a query.
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) l_run += __shfl_xor_sync(0xffffffffu, l_run, d);
    float* mine = joint + (((units & 1) * kWarps + warp) * kDecodeRows + my_q) * C::kRow;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
      mine[16 * e + (lane >> 2)] = acc[e][0] + acc[e][1];
      mine[16 * e + 8 + (lane >> 2)] = acc[e][2] + acc[e][3];
    }
    if (lane < 4) mine[D] = m_run, mine[D + 1] = l_run;
    warp_arrive(&bars->joined);
    ok = warp_wait(&bars->joined, units & 1, wait_ns, abort);
    if (!ok) break;
    for (int t = warp; t < n; t += kWarps) {
      const float* from = joint + ((units & 1) * kWarps * kDecodeRows + t) * C::kRow;
      constexpr int kStride = kDecodeRows * C::kRow;
      float o[D / 32], m_all = -INFINITY, l_all = 0.f;
#pragma unroll
      for (int y = 0; y < kWarps; ++y) m_all = fmaxf(m_all, from[y * kStride + D]);
      const float m_eff = m_all == -INFINITY ? 0.f : m_all;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
#pragma unroll
      for (int y = 0; y < kWarps; ++y) {
        const float f = ex2(from[y * kStride + D] - m_eff);
        l_all += f * from[y * kStride + D + 1];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] = fmaf(f, from[y * kStride + e * 32 + lane], o[e]);
      }
      const bool none = m_all == -INFINITY;
      const float inv = none ? 0.f : 1.f / l_all;
      const float lse2 = none ? -INFINITY : m_all + log2f(l_all);
      if (w.pieces > 1) {  // to the workspace, for the join
        float* out = p.part + plan_place(static_cast<int>(blockIdx.x), w.index) * plan_part(kDecodeRows, D);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) out[t * D + e * 32 + lane] = o[e] * inv;
        if (lane == 0) out[kDecodeRows * D + t] = lse2;
        continue;
      }
      const size_t at = (static_cast<size_t>(w.tok0 + t) * p.args.H + h) * D;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        if (O_BF16)
          static_cast<__nv_bfloat16*>(p.o)[at + e * 32 + lane] = __float2bfloat16(o[e] * inv);
        else
          static_cast<float*>(p.o)[at + e * 32 + lane] = o[e] * inv;
      }
      if (p.lse != nullptr && lane == 0)
        p.lse[static_cast<size_t>(h) * p.args.T + w.tok0 + t] = none ? -INFINITY : lse2 * 0.69314718055994531f;
    }
  }
  if (!ok && lane == 0) report_timeout(abort, p.args.status);
}

template <int D, bool O_BF16>
cudaError_t launch(const PagedAttn& a, const PlanSpace& s, int sms, bool ahead_of_tiles, const WaitCtl& wc,
                   cudaStream_t stream) {
  using C = Cfg<D>;
  PFN_cuTensorMapEncodeTiled_v12000 encode = api_tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const PageBook& b = a.book;
  CUtensorMap tm_k, tm_v, tm_r;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  auto enc = [&](CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  {
    const cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(b.page_rows), static_cast<cuuint64_t>(a.H),
                                static_cast<cuuint64_t>(b.n_pages)};
    const cuuint64_t strides[3] = {D * 2, static_cast<cuuint64_t>(b.page_rows) * D * 2,
                                   static_cast<cuuint64_t>(a.H) * b.page_rows * D * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b.page_rows < C::BK ? b.page_rows : C::BK), 1, 1};
    if (!enc(&tm_k, a.kp, 4, dims, strides, box) || !enc(&tm_v, a.vp, 4, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(a.n_r)};
    const cuuint64_t strides[2] = {D * 2, static_cast<cuuint64_t>(a.H) * D * 2};
    const cuuint32_t box[3] = {64, 1, C::BR};
    if (!enc(&tm_r, a.r, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const Params p{plan_args(a, wc.status), static_cast<const __nv_bfloat16*>(a.q), a.bias_u, a.bias_v, a.o, a.lse,
                 a.scale * 1.4426950408889634f, s.decode.cuts, s.decode.part, wc.limit_ns, ahead_of_tiles,
                 wc.inject_stall};
  auto kern = paged_decode_kernel<D, O_BF16>;
  static unsigned configured = 0;  // one bit per device ordinal < 32
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1u << dev))) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) != cudaSuccess)
      return e;
    if (dev < 32) __atomic_fetch_or(&configured, 1u << dev, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, dim3(kDecodePerSm * sms), dim3(C::kThreads), C::kSmem, stream, tm_k, tm_v, tm_r, p);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedAttn& a, const PlanSpace& s, int sms, bool ahead_of_tiles, const WaitCtl& wc,
                                cudaStream_t stream) {
  auto run = [&](auto f) { return f(a, s, sms, ahead_of_tiles, wc, stream); };
  if (a.D == 64) return a.o_bf16 ? run(launch<64, true>) : run(launch<64, false>);
  return a.o_bf16 ? run(launch<128, true>) : run(launch<128, false>);
}

}  // namespace txl
