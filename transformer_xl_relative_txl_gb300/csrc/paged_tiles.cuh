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

// The walker's unit; moves the walker on.  The first piece of a cut unit is
// noted for the kernel that joins the pieces.
__device__ __forceinline__ void publish_unit(TileWalk& walk, TileUnit* ring, uint32_t k, TileCut* cuts) {
  TileUnit u;
  u.h = walk.h;
  const int i0 = walk.qt * kTileQueries;
  u.row0 = walk.s.tok0 + i0;
  u.nq = min(kTileQueries, walk.s.n - i0);
  u.t0 = walk.p.t0;
  u.nks = walk.p.nks;
  u.d0 = walk.s.start + walk.s.rows - walk.s.n + i0;
  u.start = walk.s.start;
  u.last = walk.s.start + walk.s.rows - 1;
  u.slot = walk.s.slot;
  u.index = walk.p.index;
  u.pieces = walk.p.pieces;
  if (u.pieces > 1 && u.index == 0) cuts[blockIdx.x] = TileCut{u.row0, u.nq, u.h, u.pieces};
  u.next_h = walk.next() ? walk.h : -1;
  ring[k % kUnitRing] = u;
}

// Zeroes the rows of a landed value tile that are not live: weight 0 times a
// leftover that is no number would not be 0.  The tile's rows are shared by
// `warps` warps; the caller's proxy fence and arrival on the barrier that the
// P.V issuer waits for follow.
template <int D>
__device__ __forceinline__ void zero_dead_rows(const TileUnit& u, int t, uint8_t* stage, int warp, int warps,
                                               int lane) {
  const int x0 = t * kStepKeys;
  for (int y = warp; y < kStepKeys; y += warps) {
    if (x0 + y >= u.start && x0 + y <= u.last) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) *reinterpret_cast<uint32_t*>(stage + c * kStepKeys * 128 + y * 128 + lane * 4) = 0;
  }
}
__device__ __forceinline__ bool has_dead_rows(const TileUnit& u, int t) {
  return t * kStepKeys < u.start || t * kStepKeys + kStepKeys - 1 > u.last;
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
  float* mine = part + plan_place(static_cast<int>(blockIdx.x), u.index) * static_cast<size_t>(tile_part(D));
  float4* po = reinterpret_cast<float4*>(mine + a * D);
#pragma unroll
  for (int c = 0; c < D / 4; ++c) po[c] = make_float4(ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]);
  mine[kTileQueries * D + a] = lse2;
}

// Kernel parameters common to both.
struct TileParams {
  PageBook book;
  int log_page_rows;
  const float* bias_u;
  const float* bias_v;
  void* o;
  float* lse;
  int T, H;
  float scale_log2e;  // |scale| * log2(e)
  float qsign;        // sign of scale, folded into (q+u), (q+v)
  const PlanHead* head;
  const PlanSeq* seqs;
  const int* starts;
  TileCut* cuts;
  float* part;
  unsigned int* status;
  unsigned long long wait_ns;
};

// Tensor maps: q over {D, H, T} with a {64, 1, 128} box, the pools over
// {D, page_rows, H, n_pages} with {64, min(page_rows, 64), 1, 1}, r over
// {D, H, n_r} with {64, 1, 64}; o (bf16) over {D, H, T} with {64, 1, 32}.
struct TileMaps {
  CUtensorMap q, k, v, r, o;
};

// The loader warp of both kernels, all lanes in step: K, V and r tiles (and
// the raw q tiles) of the CTA's units in order, and the units published.
// Bars has the rings' barriers, the units and the walker (in shared memory:
// it is used once per unit, and the warp has few registers).
//
// Pages.  A 64-row tile is one box of a page, or 2 or 4 boxes of pages of 32
// or 16 rows.  Lane y (and 4 + y for V) has box y: its page id is fetched a
// tile ahead, and one TMA instruction issues all the boxes.  Boxes without a
// live row are left out; a page id out of range reads as zeros (a box outside
// its tensor) and is reported.  With one lane doing all of it the loader bound
// the kernel: 1.57 us a step at D = 64 where the softmax takes 0.8.
//
// LAG: V tiles trail the K and r tiles by so many.  A V stage is freed only
// when the P.V MMA of its step completes, after that step's softmax, while a K
// stage is free as soon as its score MMA is done; in one issue order K(t),
// R(t+1), V(t), every K load would wait behind the V stage of step t - NS and
// land just in time.  AHEAD: the raw q tile of a unit is loaded a unit ahead;
// before that of the unit after next, every queued V of a unit two or more
// back goes out, since the load waits for the (q+u), (q+v) build of the next
// unit, which waits for the epilogue of the unit before, which needs all of
// that unit's V tiles (a unit of one step would otherwise hold them behind the
// load).
template <int D, int NS, int LAG, bool AHEAD, typename Bars>
__device__ __forceinline__ void run_tile_loader(Bars* bars, const TileMaps& tm, const TileParams& p, uint8_t* sQ,
                                                uint8_t* sK, uint8_t* sV, uint8_t* sR) {
  constexpr int kChunk = kStepKeys * 128, kTile = kChunk * (D / 64), kQChunk = kTileQueries * 128;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  const uint64_t wait_ns = p.wait_ns;
  const int log_page = p.log_page_rows, log_box = min(log_page, 6);
  const int y = lane & 3;
  const bool mine = lane < 8 && y < (kStepKeys >> log_box);
  const int off = y << log_box;                  // first row of this lane's box in a tile
  const uint32_t at = static_cast<uint32_t>(off) * 128;  // its place in a stage's chunk
  if (lane == 0) {
    tma_prefetch_desc(&tm.q);
    tma_prefetch_desc(&tm.k);
    tma_prefetch_desc(&tm.v);
    tma_prefetch_desc(&tm.r);
  }
  uint32_t nQ = 0, nK = 0, nV = 0, nR = 0;
  bool ok = bars->any != 0, bad = false;
  const bool any = ok;

  auto load_q = [&](uint32_t un) {
    if (!(ok = warp_wait(&bars->q_empty, (nQ & 1) ^ 1, wait_ns, abort))) return;
    if (lane == 0) {
      const TileUnit& w = bars->units[un % kUnitRing];
      mbar_arrive_expect_tx(&bars->q_full, kQChunk * (D / 64));
#pragma unroll
      for (int c = 0; c < D / 64; ++c) tma_load_3d(sQ + c * kQChunk, &tm.q, &bars->q_full, c * 64, w.h, w.row0);
    }
    ++nQ;
  };
  auto load_r = [&](int h, int dist) {
    const int s = static_cast<int>(nR % NS);
    if (!(ok = ok && warp_wait(&bars->emptyR[s], ((nR / NS) & 1) ^ 1, wait_ns, abort))) return;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars->fullR[s], kTile);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(sR + s * kTile + c * kChunk, &tm.r, &bars->fullR[s], c * 64, h, dist);
    }
    ++nR;
  };
  // A tile of keys or values: this lane's page (-1: no live row), the row in
  // the page, the head, the tile's bytes, the unit.
  struct Tile {
    int page, x, h;
    uint32_t bytes, unit;
  };
  auto load_tile = [&](const Tile& e, uint64_t* empty, uint64_t* full, uint32_t& n, const CUtensorMap* map,
                       uint8_t* stages, bool issues) {
    const int s = static_cast<int>(n % NS);
    if (!(ok = ok && warp_wait(&empty[s], ((n / NS) & 1) ^ 1, wait_ns, abort))) return;
    if (lane == 0) mbar_arrive_expect_tx(&full[s], e.bytes);
    __syncwarp();
    if (issues && e.page >= 0) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_4d(stages + s * kTile + c * kChunk + at, map, &full[s], c * 64, e.x, e.h, e.page);
    }
    ++n;
  };
  Tile queue[LAG > 0 ? LAG : 1];  // queue[0] the oldest
  int queued = 0;
  auto issue_v = [&](const Tile& e) {
    load_tile(e, bars->emptyV, bars->fullV, nV, &tm.v, sV, lane >= 4);
  };
  auto pop_v = [&]() {
    issue_v(queue[0]);
#pragma unroll
    for (int e = 0; e + 1 < LAG; ++e) queue[e] = queue[e + 1];
    --queued;
  };

  if (AHEAD && any) load_q(0);
  for (uint32_t un = 0; any && ok; ++un) {
    const TileUnit& w = bars->units[un % kUnitRing];
    const int next_h = w.next_h, h = w.h, d0 = w.d0, start = w.start, last = w.last, tend = w.t0 + w.nks;
    const int* row = p.book.table + static_cast<size_t>(w.slot) * p.book.max_pages;
    int t = w.t0;
    if (LAG > 0)
      while (ok && queued > 0 && queue[0].unit + 2 <= un) pop_v();
    if (!ok) break;
    if (next_h >= 0) {
      if (lane == 0) publish_unit(bars->walk, bars->units, un + 1, p.cuts);
      __syncwarp();
      if (AHEAD) load_q(un + 1);
    }
    if (!AHEAD) load_q(un);
    if (!ok) break;
    auto live = [&](int tile) {
      const int x = tile * kStepKeys + off;
      return mine && x <= last && x + (1 << log_box) > start;
    };
    int id = live(t) ? row[(t * kStepKeys + off) >> log_page] : 0;
    // distance tiles -2 and -1 of the unit's first step
    load_r(h, d0 - kStepKeys * (t - 1));
    load_r(h, d0 - kStepKeys * t);
    for (; ok && t < tend; ++t) {
      const bool lv = live(t);
      Tile e;
      e.page = -1;
      if (lv) {
        const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(p.book.n_pages);
        bad |= !good;
        e.page = good ? id : p.book.n_pages;
      }
      if (t + 1 < tend) id = live(t + 1) ? row[((t + 1) * kStepKeys + off) >> log_page] : 0;
      e.bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, lv) & 0xf)) << (log_box + (D == 64 ? 7 : 8));
      e.x = (t * kStepKeys) & ((1 << log_page) - 1);  // 0 for pages of up to 64 rows
      e.h = h;
      e.unit = un;
      load_tile(e, bars->emptyK, bars->fullK, nK, &tm.k, sK, lane < 4);
      load_r(h, d0 - kStepKeys * (t + 1));
      if (LAG == 0) {
        issue_v(e);
      } else {
        if (ok && queued == LAG) pop_v();
#pragma unroll
        for (int q = 0; q < LAG; ++q)
          if (q == queued) queue[q] = e;
        ++queued;
      }
    }
    if (next_h < 0) break;
  }
  if (LAG > 0)
    while (ok && queued > 0) pop_v();
  if (bad) atomicOr(p.status, kStatusPagesBit);
  if (any && !ok && lane == 0) report_timeout(abort, p.status);
  // This warp's own copies land before the CTA may exit.
  auto drain = [&](uint64_t* full, uint32_t n, int ns) {
    for (int s = 0; s < ns && static_cast<uint32_t>(s) < n; ++s) {
      const uint32_t z = s + ((n - 1 - s) / ns) * ns;
      mbar_wait_own(&full[s], (z / ns) & 1, wait_ns);
    }
  };
  drain(&bars->q_full, nQ, 1);
  drain(bars->fullK, nK, NS);
  drain(bars->fullV, nV, NS);
  drain(bars->fullR, nR, NS);
}

cudaError_t launch_paged_tc64(const TileMaps& m, const TileParams& p, bool o_bf16, int sms, cudaStream_t stream);
cudaError_t launch_paged_tc128(const TileMaps& m, const TileParams& p, bool o_bf16, int sms, cudaStream_t stream);

}  // namespace txl
