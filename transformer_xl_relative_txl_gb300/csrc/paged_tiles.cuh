// What the two paged tensor-core kernels (D = 64 and 128) share: the unit a
// CTA's roles work on, the loads of a key tile from its pages, the zeroing of
// value rows that are not live, and the storing of results.
//
// The loader warp finds the CTA's units (paged_plan.cuh) and publishes them in
// a ring in shared memory before it loads their queries; every other role
// reads a unit after a barrier that follows that load.  It publishes up to 32
// at a time, once fewer than two behind the one at hand are known, and no role
// is more than four units behind it: a ring of 64 never overtakes a reader.
#pragma once

#include "paged_plan.cuh"
#include "relattn_tc_common.cuh"
#include "txl_device.cuh"

namespace txl {

constexpr int kUnitRing = 64;

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

// One warp.  The CTA's next units into the ring, behind the `known` that it
// has: how many there are then.  A unit is whole once the one behind it is
// known, or known not to be (*ended).  The first piece of a cut unit is noted
// for the kernel that joins the pieces.
template <typename Bars>
__device__ __forceinline__ uint32_t publish_units(Bars* bars, const PlanArgs& args, uint32_t known, PlanCut* cuts,
                                                  bool* ended) {
  const int lane = threadIdx.x & 31;
  PlanFound f{};
  const int found = plan_batch<TileUnits>(args, &bars->plan, known == 0, &f, ended);
  int next_h = __shfl_down_sync(0xffffffffu, f.h, 1);
  if (lane == found - 1) next_h = -1;
  if (lane < found) {
    TileUnit& u = bars->units[(known + lane) % kUnitRing];
    const int i0 = f.qt * kTileQueries;
    u.h = f.h;
    u.row0 = f.s.tok0 + i0;
    u.nq = min(kTileQueries, f.s.n - i0);
    u.t0 = f.p.t0;
    u.nks = f.p.nks;
    u.d0 = f.s.start + f.s.rows - f.s.n + i0;
    u.start = f.s.start;
    u.last = f.s.start + f.s.rows - 1;
    u.slot = f.s.slot;
    u.index = f.p.index;
    u.pieces = f.p.pieces;
    u.next_h = next_h;
    if (f.p.pieces > 1 && f.p.index == 0) cuts[blockIdx.x] = PlanCut{u.row0, u.nq, u.h, u.pieces};
  }
  if (lane == 0 && known > 0) bars->units[(known - 1) % kUnitRing].next_h = found > 0 ? f.h : -1;
  __syncwarp();
  return known + found;
}

// Bit k: column k of 32 lies in low .. lim.  (Masking by bits, the test of a
// column is short code for a block that most steps pass by: with two compares
// a column, and the columns in a line, 12% longer for 22 sequences of 512 tokens
// over 512 rows, though almost no step runs it.)
__device__ __forceinline__ uint32_t visible_columns(int low, int lim) {
  const uint32_t upto = lim < 0 ? 0u : 0xffffffffu >> max(31 - lim, 0);
  const uint32_t from = low > 31 ? 0u : 0xffffffffu << max(low, 0);
  return upto & from;
}

// The P.V issuer's warp: zeroes the rows of the landed value tile t that are
// not live: weight 0 times a leftover that is no number would not be 0.  (In the
// softmax warps, behind their step's weights, the code alone cost their loop
// 7%, though almost no step runs it.)
template <int D>
__device__ __forceinline__ void zero_dead_rows(int start, int last, int t, uint8_t* stage, int lane) {
  const int x0 = t * kStepKeys;
  if (start <= x0 && x0 + kStepKeys - 1 <= last) return;
#pragma unroll 1
  for (int y = lane >> 3; y < kStepKeys; y += 4) {
    if (x0 + y >= start && x0 + y <= last) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      *reinterpret_cast<uint4*>(stage + c * kStepKeys * 128 + y * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// The score products' bias terms: (q + u) . k = q . k + u . k, and q . k has exact
// operands.  u . k is a number a key, the same for every query, so the issuer's
// warp computes it from the landed tile, u in two bf16 parts, and appends it to
// the tile in three (24 bits), which one more product of 16 columns multiplies
// by ones.  (q + u rounded to bf16 is off by 1.65e-3 (rms) of a score's content
// part, as much as the output's own rounding.  Measured, us of 22 sequences of
// 512 tokens over 512 rows, D = 64, and of 8 of 768 over 768, D = 128, 8 heads: 104
// and 110; as products of their own with u's parts repeated for 128 rows, 114 and
// 148, with one part only 101 and 124.)
//
// Per stage of the ring, 2 KB: the 64 rows' first 8 columns, 16 bytes a row, then
// as many zeros; behind the stages 8 rows of ones (three columns), which all of
// the 128 rows read: a stride of 0 between groups of 8 in the descriptor.
constexpr int kBiasStage = 2 * kStepKeys * 16;
constexpr int kBiasOnes = 256;

// One warp's.
template <int D, int STAGES>
struct BiasTerm {
  static constexpr int kBytes = STAGES * kBiasStage + kBiasOnes;
  uint8_t* area;
  uint32_t u[D / 16][2];  // right-hand fragments: column n of 8 has part n % 2 of u

  // At the kernel's head: the parts of the area that stay.
  __device__ __forceinline__ explicit BiasTerm(uint8_t* at) : area(at) {
    constexpr int kOnes = STAGES * kBiasStage / 16;
    for (int e = threadIdx.x & 31; e < kBytes / 16; e += 32)
      reinterpret_cast<uint4*>(area)[e] =
          e >= kOnes && e < kOnes + 8 ? make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncwarp();
  }
  __device__ __forceinline__ void load(const float* bias, int h) {
    const int lane = threadIdx.x & 31;
    const float* at = bias + static_cast<size_t>(h) * D + 2 * (lane & 3);
#pragma unroll
    for (int e = 0; e < D / 8; ++e) {
      const float x = __ldg(at + 8 * e), y = __ldg(at + 8 * e + 1);
      const uint32_t hi = pack_bf16x2(x, y);
      u[e / 2][e % 2] = lane >> 2 & 1 ? pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi)) : hi;
    }
  }
  // The terms of a tile's 64 rows (128-byte swizzle): of each 16 rows, lane l has
  // those of rows l / 4 and l / 4 + 8, and puts down the (l % 4)-th 16's.
  // (As multiply-adds 119 us at D = 128 in a loop, 194 in a line: the softmax's
  // code pushes it out of the instruction cache between any two tiles.)
  __device__ __forceinline__ void append(const uint8_t* tile, int s) const {
    const int lane = threadIdx.x & 31, r16 = lane & 15, half = lane >> 4;
    float mine[2] = {0.f, 0.f};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        uint32_t a[4];
        ldsm4(smem_u32(tile) + (e / 4) * kStepKeys * 128 + (16 * y + r16) * 128 +
                  ((((e % 4) * 2 + half) ^ (r16 & 7)) << 4), a);
        mma16816(z, a, u[e][0], u[e][1]);
      }
      if ((lane & 3) == y) mine[0] = z[0] + z[1], mine[1] = z[2] + z[3];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // (A term that is not finite has no further parts.)
      const float hi = __bfloat162float(__float2bfloat16(mine[i]));
      const float rest = isfinite(hi) ? mine[i] - hi : 0.f;
      const uint32_t two = pack_bf16x2(hi, rest);
      *reinterpret_cast<uint4*>(area + s * kBiasStage + (16 * (lane & 3) + 8 * i + (lane >> 2)) * 16) =
          make_uint4(two, pack_bf16x2(rest - bf16_hi(two), 0.f), 0u, 0u);
    }
    fence_proxy_async_smem();
    __syncwarp();
  }
  __device__ __forceinline__ uint64_t ones_desc() const {
    return sdesc_plain(smem_u32(area + STAGES * kBiasStage), kBiasOnes / 2, 0);
  }
  __device__ __forceinline__ uint64_t term_desc() const { return sdesc_plain(smem_u32(area), kBiasStage / 2, 128); }
};

// One thread: D[128 x 64] = q B^T + the bias term, of a tile B of 64 rows.  q, b:
// descriptors (64-dimension chunks kTileQueries and kStepKeys rows apart), ones,
// term: of the bias area.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t q, uint64_t b, uint64_t ones, uint64_t term,
                                           uint32_t id) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_ss(d, q + (((kk / 4) * kTileQueries * 128 + (kk % 4) * 32) >> 4),
           b + (((kk / 4) * kStepKeys * 128 + (kk % 4) * 32) >> 4), id, kk > 0);
  mma_ss(d, ones, term, id, 1);
}

// Per-lane window shift in fp32: lo, hi hold the window X[0..63]; out[k] =
// X[lane + 32 - k], k = 0..31, the distance value of key column k.  (In bf16
// pairs, packed and unpacked, it is 102 selects of 372 shorter, less the adds
// that take two columns at a time here; it rounds the distance part to 2^-8.)
__device__ __forceinline__ void window_shift_f32(const uint32_t (&lo)[32], const uint32_t (&hi)[32], int lane,
                                                 uint32_t (&out)[32]) {
  uint32_t R[63];
#pragma unroll
  for (int i = 0; i < 63; ++i) R[i] = i < 31 ? lo[i + 1] : hi[i - 31];
  const bool b16 = lane & 16, b8 = lane & 8, b4 = lane & 4, b2 = lane & 2, b1 = lane & 1;
#pragma unroll
  for (int j = 0; j < 47; ++j) R[j] = b16 ? R[j + 16] : R[j];
#pragma unroll
  for (int j = 0; j < 39; ++j) R[j] = b8 ? R[j + 8] : R[j];
#pragma unroll
  for (int j = 0; j < 35; ++j) R[j] = b4 ? R[j + 4] : R[j];
#pragma unroll
  for (int j = 0; j < 33; ++j) R[j] = b2 ? R[j + 2] : R[j];
#pragma unroll
  for (int k = 0; k < 32; ++k) out[k] = b1 ? R[32 - k] : R[31 - k];
}
// x[k] = s[k] + d[k]
__device__ __forceinline__ void add_columns(const uint32_t (&s)[32], const uint32_t (&d)[32], float* x) {
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    const float2 y = __fadd2_rn(make_float2(__uint_as_float(s[2 * n]), __uint_as_float(s[2 * n + 1])),
                                make_float2(__uint_as_float(d[2 * n]), __uint_as_float(d[2 * n + 1])));
    x[2 * n] = y.x;
    x[2 * n + 1] = y.y;
  }
}

// A pair of weights as two bf16 pairs, hi + lo.
__device__ __forceinline__ void split_weights(float2 e, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(e.x, e.y);
  const float2 rest = __ffma2_rn(make_float2(bf16_lo(hi), bf16_hi(hi)), make_float2(-1.f, -1.f), e);
  lo = pack_bf16x2(rest.x, rest.y);
}

// Results of a unit, o normalised by its own sum, lse2 its log2-domain lse
// (-inf: no visible key).  A whole unit's go to the output, rows past its
// queries are not written; a piece's go to the workspace, joined by the kernel
// behind this one (paged_join.cu).  (With the last piece to arrive joining in
// this kernel, its warps held up the CTA's softmax: half as long again for 22
// sequences of 512 tokens over 512 rows, 8 heads, where every CTA has two
// pieces.)
__device__ __forceinline__ float* piece_of(const TileUnit& u, float* part, int D) {
  return part + plan_place(static_cast<int>(blockIdx.x), u.index) * static_cast<size_t>(plan_part(kTileQueries, D));
}
__device__ __forceinline__ void store_lse(const TileUnit& u, int a, float lse2, float* lse, float* part, int T, int D) {
  if (u.pieces > 1)
    piece_of(u, part, D)[kTileQueries * D + a] = lse2;
  else if (a < u.nq && lse != nullptr)
    lse[static_cast<size_t>(u.h) * T + u.row0 + a] = lse2 == -INFINITY ? -INFINITY : lse2 * 0.69314718055994531f;
}
// Columns 32 oc .. 32 oc + 31 of row a.
template <int D, bool O_BF16>
__device__ __forceinline__ void store_columns(const TileUnit& u, int a, int oc, const float (&ov)[32], void* o,
                                              float* part, int H) {
  float* to = nullptr;
  if (u.pieces > 1) {
    to = piece_of(u, part, D) + a * D;
  } else {
    if (a >= u.nq) return;
    const size_t at = (static_cast<size_t>(u.row0 + a) * H + u.h) * D;
    if (O_BF16) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o) + at) + 4 * oc;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        dst[c] = make_uint4(pack_bf16x2(ov[8 * c], ov[8 * c + 1]), pack_bf16x2(ov[8 * c + 2], ov[8 * c + 3]),
                            pack_bf16x2(ov[8 * c + 4], ov[8 * c + 5]), pack_bf16x2(ov[8 * c + 6], ov[8 * c + 7]));
      return;
    }
    to = static_cast<float*>(o) + at;
  }
  float4* dst = reinterpret_cast<float4*>(to) + 8 * oc;
#pragma unroll
  for (int c = 0; c < 8; ++c) dst[c] = make_float4(ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]);
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
  bool negative;      // of scale: the score products negate their A operand
  PlanCut* cuts;
  float* part;
  unsigned long long wait_ns;
  int inject_stall;
};

// Tensor maps: q over {D, H, T} with a {64, 1, 128} box, the pools over
// {D, page_rows, H, n_pages} with {64, min(page_rows, 64), 1, 1}, r over
// {D, n_r, H, 1} with {64, 64, 1, 1}; o (bf16) over {D, H, T} with {64, 1, 32}.
struct TileMaps {
  CUtensorMap q, k, v, r, o;
};

// The loader warp of both kernels: K, V and r tiles (and the raw q tiles) of
// the CTA's units in order, and the units published.  It has the CTA's barrier
// behind the first units; bars->any says whether there is one.
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
// TRAIL: a V tile goes out with the K tile of the step behind.  A V stage is
// freed only when the P.V MMA of its step completes, after that step's softmax,
// while a K stage is free as soon as its score MMA is done; with V(t) beside
// K(t), K would wait for the P.V of step t - NS and land just in time (D = 128,
// two stages: 15% longer for 152 units of 100 steps; at D = 64, with four stages, a
// V tile that trails takes 6% longer).  The q tile of a unit is
// loaded ahead of its first step, into the one of two buffers that the score
// products of the unit before the last have read.
//
// STALL: the kernels' instances for the test hook, in which the loader of even
// CTAs, and the P.V issuer of odd ones, stops behind its first unit's first
// step.  (As a test of a parameter it cost the D = 64 kernel 2 to 5%.)
template <int D, int NS, bool TRAIL, bool STALL, typename Bars>
__device__ __forceinline__ void run_tile_loader(Bars* bars, const TileMaps& tm, const TileParams& p, uint8_t* sQ,
                                                uint8_t* sK, uint8_t* sV, uint8_t* sR) {
  static_assert((NS & (NS - 1)) == 0, "stage arithmetic");
  constexpr int kChunk = kStepKeys * 128, kTile = kChunk * (D / 64), kQChunk = kTileQueries * 128;
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
  uint32_t loaded = 0;  // q tiles so far
  bool ok = true, bad = false;

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
    const uint32_t s = un & 1;
    if (!(ok = warp_wait(&bars->q_empty[s], ((un >> 1) & 1) ^ 1, p.wait_ns, abort))) return;
    if (lane == 0) {
      const TileUnit& w = bars->units[un % kUnitRing];
      mbar_arrive_expect_tx(&bars->q_full[s], kQChunk * (D / 64));
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(sQ + (s * (D / 64) + c) * kQChunk, &tm.q, &bars->q_full[s], c * 64, w.h, w.row0);
    }
    loaded = un + 1;
  };
  // A tile of keys: this lane's page (-1: no live row), the row in the page,
  // the head, the tile's bytes.
  struct Tile {
    int page, x, h;
    uint32_t bytes;
  };
  Tile held{};  // the V tile that trails
  bool holds = false;
  auto release = [&]() {
    if (holds) issue(is_v, held.page, held.x, held.h, held.bytes);
    holds = false;
  };

  // `known` units are published, all whole but the last (`ended`: the last
  // too); the tiles of unit `un`, of which t is the next, are under way.
  uint32_t known = 0, un = 0xffffffffu;
  bool ended = false, begun = false;
  const bool stall = STALL && blockIdx.x % 2 == 0;
  int h = 0, d0 = 0, start = 0, last = 0, t = 0, t0 = 0, tend = 0, id = 0;
  const int* row = nullptr;
  auto live = [&](int tile) {
    const int x = tile * kStepKeys + off;
    return boxed && x <= last && x + (1 << log_box) > start;
  };
  for (;;) {
    // Unit un + 1 whole.
    while (!ended && known < un + 3) known = publish_units(bars, p.args, known, p.cuts, &ended);
    if (!begun) {
      if (known > 0) {  // the first tile's pages, on their way meanwhile
        const TileUnit& w = bars->units[0];
        const int x = w.t0 * kStepKeys + off;
        if (boxed && x <= w.last && x + (1 << log_box) > w.start)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(
              p.args.book.table + static_cast<size_t>(w.slot) * p.args.book.max_pages + (x >> log_page)));
      }
      begun = true;
      if (lane == 0) bars->any = known > 0;
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      if (known == 0) break;
    }
    // Tiles, up to a unit's first step.
    bool head = false, done = false;
    while (ok && !head) {
      if (t == tend) {  // the next unit
        if (++un == known || (stall && un > 0)) {
          done = true;
          break;
        }
        load_q(un);
        if (!ok) break;
        const TileUnit& w = bars->units[un % kUnitRing];
        h = w.h, d0 = w.d0, start = w.start, last = w.last, t0 = w.t0, tend = t0 + (stall ? 1 : w.nks);
        row = p.args.book.table + static_cast<size_t>(w.slot) * p.args.book.max_pages;
        id = live(t0) ? row[(t0 * kStepKeys + off) >> log_page] : 0;
        t = t0 - 2;  // its first step's other distance tiles
      }
      const bool step = t >= t0;
      const bool lv = step && live(t);
      Tile e;
      e.page = -1;
      if (lv) {
        const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(p.args.book.n_pages);
        bad |= !good;
        e.page = good ? id : p.args.book.n_pages;
      }
      if (step && t + 1 < tend) id = live(t + 1) ? row[((t + 1) * kStepKeys + off) >> log_page] : 0;
      e.bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, lv) & 0xf)) << (log_box + (D == 64 ? 7 : 8));
      e.x = (t * kStepKeys) & ((1 << log_page) - 1);  // 0 for pages of up to 64 rows
      e.h = h;
      const bool has_v = step && (!TRAIL || holds);
      const Tile& v = TRAIL ? held : e;
      issue(is_r || (is_k && step) || (is_v && has_v), is_r ? 0 : (is_v ? v.page : e.page),
            is_r ? d0 - kStepKeys * (t + 1) : (is_v ? v.x : e.x), is_v ? v.h : h,
            is_r ? static_cast<uint32_t>(kTile) : (is_v ? v.bytes : e.bytes));
      if (TRAIL && step) {
        held = e;
        holds = true;
      }
      head = t == t0;
      ++t;
    }
    if (!ok || done) break;
  }
  if (TRAIL && ok) release();
  if (bad) atomicOr(p.args.status, kStatusPagesBit);
  if (!ok && lane == 0) report_timeout(abort, p.args.status);
  // This warp's own copies land before the CTA may exit.
  for (uint32_t un = loaded > 2 ? loaded - 2 : 0; un < loaded; ++un)
    mbar_wait_own(&bars->q_full[un & 1], (un >> 1) & 1, p.wait_ns);
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
