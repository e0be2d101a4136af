// What the two paged tensor-core kernels (D = 64 and 128) share: the unit a
// CTA's roles work on, the loads of a key tile from its pages, the zeroing of
// value rows that are not live, and the joining of pieces.
//
// The loader warp's first lane walks the CTA's units (paged_plan.cuh) and
// publishes each in a ring in shared memory before the barrier that announces
// the unit's queries; every other role reads a unit after a barrier that
// follows that one.  A unit is published once the operands of the unit before
// it are built, which is at the earliest while the unit before that runs its
// first step, so no role is more than three units behind.
#pragma once

#include "paged_plan.cuh"
#include "relattn_tc_common.cuh"
#include "txl_device.cuh"

namespace txl {

constexpr int kUnitRing = 8;

struct TileUnit {
  int h;               // head
  int row0, nq;        // first row of q and o, queries
  int t0, nks;         // key steps, from the slot's first page
  int d0;              // page row of query 0: query a sees rows start .. d0 + a at distance d0 + a - row
  int start, last;     // live page rows
  int slot;
  int index, pieces;
  int next_h;          // head of the CTA's next unit, -1: none
};

// One warp.  The walker's unit into the ring, the walker to the next; the first
// piece of a cut unit is noted for the kernel that joins the pieces.
template <typename Bars>
__device__ __forceinline__ void publish_unit(Bars* bars, const PlanArgs& args, uint32_t k, PlanCut* cuts) {
  const bool lead = (threadIdx.x & 31) == 0;
  TileUnit& u = bars->units[k % kUnitRing];
  // The walker works in registers: in place, each of its dependent steps would
  // cost a shared-memory latency.
  TileWalk walk = bars->walk;
  const int i0 = walk.qt * kTileQueries;
  if (lead) {
    const int nq = min(kTileQueries, walk.s.n - i0);
    u.h = walk.h;
    u.row0 = walk.s.tok0 + i0;
    u.nq = nq;
    u.t0 = walk.p.t0;
    u.nks = walk.p.nks;
    u.d0 = walk.s.start + walk.s.rows - walk.s.n + i0;
    u.start = walk.s.start;
    u.last = walk.s.start + walk.s.rows - 1;
    u.slot = walk.s.slot;
    u.index = walk.p.index;
    u.pieces = walk.p.pieces;
    if (walk.p.pieces > 1 && walk.p.index == 0)
      cuts[blockIdx.x] = PlanCut{walk.s.tok0 + i0, nq, walk.h, walk.p.pieces};
  }
  PlanStep step = walk.next();
  while (step == kPlanFill) {
    const int count = plan_fill<TileWalk>(args, &bars->plan);
    step = walk.filled(count, bars->plan.raw < args.n);
  }
  __syncwarp();  // every lane has read the walker
  if (lead) {
    u.next_h = step == kPlanUnit ? walk.h : -1;
    bars->walk = walk;
  }
  __syncwarp();
}

// All threads of the CTA, behind grid_dep_wait: the division of the work; the
// warp `loader` then publishes the CTA's first unit, if it has one (bars->any),
// which the barrier that the caller has next makes known.
template <typename Bars>
__device__ __forceinline__ void begin_units(Bars* bars, const PlanArgs& args, PlanCut* cuts, int loader) {
  if (threadIdx.x == 0) cuts[blockIdx.x] = PlanCut{0, 0, 0, 0};
  plan_begin<TileWalk>(args, static_cast<int>(gridDim.x), &bars->plan);
  if (static_cast<int>(threadIdx.x >> 5) != loader) return;
  const bool lead = (threadIdx.x & 31) == 0;
  PlanStep step = kPlanEnd;
  if (static_cast<int>(blockIdx.x) < bars->plan.ctas) {
    TileWalk walk;
    int count = plan_fill<TileWalk>(args, &bars->plan);
    step = walk.begin(bars->plan.seqs, count, bars->plan.raw < args.n, bars->plan.total, bars->plan.ctas, args.H,
                      static_cast<int>(blockIdx.x));
    while (step == kPlanFill) {
      count = plan_fill<TileWalk>(args, &bars->plan);
      step = walk.filled(count, bars->plan.raw < args.n);
    }
    if (lead) bars->walk = walk;
    __syncwarp();
  }
  if (lead) bars->any = step == kPlanUnit ? 1 : 0;
  if (step == kPlanUnit) publish_unit(bars, args, 0, cuts);
}

// Zeroes the rows of a landed value tile that are not live: weight 0 times a
// leftover that is no number would not be 0.  The tile's rows are shared by
// `warps` warps; the caller's proxy fence and arrival on the barrier that the
// P.V issuer waits for follow.
template <int D>
__device__ __forceinline__ void zero_dead_rows(int start, int last, int t, uint8_t* stage, int warp, int warps,
                                               int lane) {
  const int x0 = t * kStepKeys;
  for (int y = warp; y < kStepKeys; y += warps) {
    if (x0 + y >= start && x0 + y <= last) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) *reinterpret_cast<uint32_t*>(stage + c * kStepKeys * 128 + y * 128 + lane * 4) = 0;
  }
}

// Row `a` of a unit (lane `lane` of quadrant `quad`), o normalised by its own
// sum, lse2 its log2-domain lse (-inf: no visible key), to the output; rows
// past the unit's queries are not written.
template <int D, bool O_BF16>
__device__ __forceinline__ void store_row(const TileUnit& u, int a, const float (&ov)[D], float lse2, void* o,
                                          float* lse, int T, int H) {
  if (a >= u.nq) return;
  const size_t at = (static_cast<size_t>(u.row0 + a) * H + u.h) * D;
  if (O_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o) + at);
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      dst[c] = make_uint4(pack_bf16x2(ov[8 * c], ov[8 * c + 1]), pack_bf16x2(ov[8 * c + 2], ov[8 * c + 3]),
                          pack_bf16x2(ov[8 * c + 4], ov[8 * c + 5]), pack_bf16x2(ov[8 * c + 6], ov[8 * c + 7]));
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(o) + at);
#pragma unroll
    for (int c = 0; c < D / 4; ++c) dst[c] = make_float4(ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]);
  }
  if (lse != nullptr)
    lse[static_cast<size_t>(u.h) * T + u.row0 + a] = lse2 == -INFINITY ? -INFINITY : lse2 * 0.69314718055994531f;
}

// A piece's row goes to the workspace, joined by the kernel behind this one
// (paged_join.cu).  (With the last piece to arrive joining in this kernel, its
// warps held up the CTA's softmax: 131 us instead of 90 for 22 sequences of
// 512 tokens over 512 rows, 8 heads, where every CTA has two pieces.)
template <int D>
__device__ __forceinline__ void store_piece(const TileUnit& u, int a, const float (&ov)[D], float lse2, float* part) {
  float* mine = part + plan_place(static_cast<int>(blockIdx.x), u.index) * static_cast<size_t>(plan_part(kTileQueries, D));
  float4* po = reinterpret_cast<float4*>(mine + a * D);
#pragma unroll
  for (int c = 0; c < D / 4; ++c) po[c] = make_float4(ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]);
  mine[kTileQueries * D + a] = lse2;
}

// Kernel parameters common to both.
struct TileParams {
  PlanArgs args;
  int log_page_rows;
  const float* bias_u;
  const float* bias_v;
  void* o;
  float* lse;
  float scale_log2e;  // |scale| * log2(e)
  float qsign;        // sign of scale, folded into (q+u), (q+v)
  PlanCut* cuts;
  float* part;
  unsigned long long wait_ns;
};

// Tensor maps: q over {D, H, T} with a {64, 1, 128} box, the pools over
// {D, page_rows, H, n_pages} with {64, min(page_rows, 64), 1, 1}, r over
// {D, n_r, H, 1} with {64, 64, 1, 1}; o (bf16) over {D, H, T} with {64, 1, 32}.
struct TileMaps {
  CUtensorMap q, k, v, r, o;
};

// The loader warp of both kernels: K, V and r tiles (and the raw q tiles) of
// the CTA's units in order, and the units published.  Bars has the rings'
// barriers, the units and the walker (in shared memory: it is used once per
// unit, and the warp has few registers).
//
// The lanes share a step's work: lanes 0-3 have the boxes of its K tile, 4-7
// those of a V tile, 8 its r tile.  A 64-row tile of keys is one box of a page,
// or 2 or 4 boxes of pages of 32 or 16 rows; a lane fetches its box's page id a
// tile ahead.  Lanes 0, 4 and 8 wait for their stages at the same time, then
// one instruction arms the three barriers and one issues every box.  (One lane
// doing all in turn took 2900 cycles a step at D = 64, all lanes doing it in
// turn 2500; the softmax takes 1460.)  Boxes without a live row are left out; a
// page id out of range reads as zeros (a box outside its tensor) and is
// reported.
//
// LAG: V tiles trail the K and r tiles by so many.  A V stage is freed only
// when the P.V MMA of its step completes, after that step's softmax, while a K
// stage is free as soon as its score MMA is done; with V(t) beside K(t), K
// would wait for the P.V of step t - NS and land just in time (D = 128: 158 us
// instead of 131 for 152 units of 100 steps).  AHEAD: the raw q tile of a unit
// is loaded a unit ahead, and before that of the unit after next every queued V
// of a unit two or more back goes out, since the load waits for the (q+u),
// (q+v) build of the next unit, which waits for the epilogue of the unit
// before, which needs all of that unit's V tiles (a unit of one step would
// otherwise hold them behind the load).  Without AHEAD the build comes at the
// end of a unit's steps, which may wait for its last V (rows that are not
// live), and the next unit's r tiles wait for the build: the queue is emptied
// at each unit.
template <int D, int NS, int LAG, bool AHEAD, typename Bars>
__device__ __forceinline__ void run_tile_loader(Bars* bars, const TileMaps& tm, const TileParams& p, uint8_t* sQ,
                                                uint8_t* sK, uint8_t* sV, uint8_t* sR) {
  static_assert((NS & (NS - 1)) == 0 && LAG <= 2, "stage arithmetic, queue");
  constexpr int kChunk = kStepKeys * 128, kTile = kChunk * (D / 64), kQChunk = kTileQueries * 128;
  constexpr uint32_t kHold = AHEAD ? 2 : 1;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  const int log_page = p.log_page_rows, log_box = min(log_page, 6);
  const bool is_k = lane < 4, is_v = lane >= 4 && lane < 8, is_r = lane == 8, leads = (lane & 3) == 0 && lane <= 8;
  const bool boxed = lane < 8 && (lane & 3) < (kStepKeys >> log_box);
  const int off = (lane & 3) << log_box;  // first row of this lane's box in a tile
  uint64_t* const empty = is_v ? bars->emptyV : (is_r ? bars->emptyR : bars->emptyK);
  uint64_t* const full = is_v ? bars->fullV : (is_r ? bars->fullR : bars->fullK);
  uint8_t* const stages = is_v ? sV : (is_r ? sR : sK);
  const CUtensorMap* const map = is_v ? &tm.v : (is_r ? &tm.r : &tm.k);
  uint8_t* const mine = stages + (is_r ? 0 : off * 128);
  if (lane <= 8 && leads) tma_prefetch_desc(map);
  uint32_t n = 0;   // tiles of this lane's ring so far
  uint32_t nQ = 0;  // q tiles so far
  const bool any = bars->any != 0;
  bool ok = any, bad = false;

  // One tile of each ring whose lanes are `active`.
  auto issue = [&](bool active, int page, int x, int h, uint32_t bytes) {
    const uint32_t s = n & (NS - 1);
    const bool lead = active && leads;
    uint64_t since = 0;
    for (uint32_t tries = 1;; ++tries) {
      const bool done = !lead || mbar_try_wait(&empty[s], ((n / NS) & 1) ^ 1);
      if (__all_sync(0xffffffffu, done)) break;
      if ((tries & 15) == 0) {
        const uint64_t now = global_timer_ns();
        if (since == 0) since = now;
        if (__any_sync(0xffffffffu, *abort != 0 || now - since > p.wait_ns)) {
          ok = false;
          return;
        }
      }
    }
    if (lead) mbar_arrive_expect_tx(&full[s], bytes);
    __syncwarp();
    if (active && page >= 0) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) tma_load_4d(mine + s * kTile + c * kChunk, map, &full[s], c * 64, x, h, page);
    }
    if (active) ++n;
  };
  auto load_q = [&](uint32_t un) {
    if (!(ok = warp_wait(&bars->q_empty, (nQ & 1) ^ 1, p.wait_ns, abort))) return;
    if (lane == 0) {
      const TileUnit& w = bars->units[un % kUnitRing];
      mbar_arrive_expect_tx(&bars->q_full, kQChunk * (D / 64));
#pragma unroll
      for (int c = 0; c < D / 64; ++c) tma_load_3d(sQ + c * kQChunk, &tm.q, &bars->q_full, c * 64, w.h, w.row0);
    }
    ++nQ;
  };
  // V tiles that wait their turn, the oldest in v0: this lane's page (-1: no
  // live row), the row in the page, the head, the tile's bytes, the unit.
  struct Tile {
    int page, x, h;
    uint32_t bytes, unit;
  };
  Tile v0{}, v1{};
  int queued = 0;
  auto flush_v = [&](uint32_t upto) {  // of units up to `upto`
    while (ok && queued > 0 && v0.unit <= upto) {
      issue(is_v, v0.page, v0.x, v0.h, v0.bytes);
      v0 = v1;
      --queued;
    }
  };

  if (AHEAD && any) load_q(0);
  for (uint32_t un = 0; ok; ++un) {
    const TileUnit& w = bars->units[un % kUnitRing];
    const int next_h = w.next_h, h = w.h, d0 = w.d0, start = w.start, last = w.last, tend = w.t0 + w.nks;
    const int* row = p.args.book.table + static_cast<size_t>(w.slot) * p.args.book.max_pages;
    int t = w.t0;
    if (LAG > 0 && un >= kHold) flush_v(un - kHold);
    if (!ok) break;
    if (next_h >= 0) {
      publish_unit(bars, p.args, un + 1, p.cuts);
      if (AHEAD) load_q(un + 1);
    }
    if (!AHEAD) load_q(un);
    if (!ok) break;
    auto live = [&](int tile) {
      const int x = tile * kStepKeys + off;
      return boxed && x <= last && x + (1 << log_box) > start;
    };
    int id = live(t) ? row[(t * kStepKeys + off) >> log_page] : 0;
    // distance tiles -2 and -1 of the unit's first step
    issue(is_r, 0, d0 - kStepKeys * (t - 1), h, kTile);
    if (ok) issue(is_r, 0, d0 - kStepKeys * t, h, kTile);
    for (; ok && t < tend; ++t) {
      const bool lv = live(t);
      Tile e;
      e.page = -1;
      if (lv) {
        const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(p.args.book.n_pages);
        bad |= !good;
        e.page = good ? id : p.args.book.n_pages;
      }
      if (t + 1 < tend) id = live(t + 1) ? row[((t + 1) * kStepKeys + off) >> log_page] : 0;
      e.bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, lv) & 0xf)) << (log_box + (D == 64 ? 7 : 8));
      e.x = (t * kStepKeys) & ((1 << log_page) - 1);  // 0 for pages of up to 64 rows
      e.h = h;
      e.unit = un;
      const bool has_v = LAG == 0 || queued == LAG;
      const Tile& v = LAG == 0 ? e : v0;
      issue(is_k || is_r || (is_v && has_v), is_r ? 0 : (is_v ? v.page : e.page),
            is_r ? d0 - kStepKeys * (t + 1) : (is_v ? v.x : e.x), is_v ? v.h : h,
            is_r ? static_cast<uint32_t>(kTile) : (is_v ? v.bytes : e.bytes));
      if (LAG > 0) {
        if (has_v) {
          v0 = v1;
          --queued;
        }
        if (queued == 0)
          v0 = e;
        else
          v1 = e;
        ++queued;
      }
    }
    if (next_h < 0) break;
  }
  if (LAG > 0) flush_v(0xffffffffu);
  if (bad) atomicOr(p.args.status, kStatusPagesBit);
  if (any && !ok && lane == 0) report_timeout(abort, p.args.status);
  // This warp's own copies land before the CTA may exit.
  if (nQ > 0) mbar_wait_own(&bars->q_full, (nQ - 1) & 1, p.wait_ns);
  if (leads)
    for (uint32_t s = 0; s < NS && s < n; ++s) {
      const uint32_t z = s + ((n - 1 - s) / NS) * NS;
      mbar_wait_own(&full[s], (z / NS) & 1, p.wait_ns);
    }
  __syncwarp();
}

cudaError_t launch_paged_tc64(const TileMaps& m, const TileParams& p, bool o_bf16, int sms, cudaStream_t stream);
cudaError_t launch_paged_tc128(const TileMaps& m, const TileParams& p, bool o_bf16, int sms, cudaStream_t stream);

}  // namespace txl
