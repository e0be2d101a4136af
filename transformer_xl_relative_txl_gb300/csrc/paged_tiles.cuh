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
  int first, index, pieces;
  int next_h;          // head of the CTA's next unit, -1: none
};

// The walker's unit; moves the walker on.
__device__ __forceinline__ void publish_unit(TileWalk& walk, TileUnit* ring, uint32_t k) {
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
  u.first = walk.p.first;
  u.index = walk.p.index;
  u.pieces = walk.p.pieces;
  u.next_h = walk.next() ? walk.h : -1;
  ring[k % kUnitRing] = u;
}

// The pages of a 64-row key tile, in boxes of min(page_rows, 64) rows.
// (Page rows stay below 2^30, so a tile's row numbers are ints.)
struct TilePages {
  int id[4];  // of the boxes that hold a live row
};
struct PageMap {
  const int* table;
  int max_pages, n_pages, log_page, log_box, boxes;
  __device__ __forceinline__ PageMap(const PageBook& b, int log_page_rows)
      : table(b.table), max_pages(b.max_pages), n_pages(b.n_pages), log_page(log_page_rows),
        log_box(min(log_page_rows, 6)), boxes(kStepKeys >> min(log_page_rows, 6)) {}
  // Whether box y of tile t holds a live row.
  __device__ __forceinline__ bool live(const TileUnit& u, int t, int y) const {
    const int x = t * kStepKeys + (y << log_box);
    return y < boxes && x <= u.last && x + (1 << log_box) > u.start;
  }
  __device__ __forceinline__ TilePages pages(const TileUnit& u, int t) const {
    const int* row = table + static_cast<size_t>(u.slot) * max_pages;
    TilePages p;
#pragma unroll
    for (int y = 0; y < 4; ++y) p.id[y] = live(u, t, y) ? row[(t * kStepKeys + (y << log_box)) >> log_page] : 0;
    return p;
  }
};

// Loads tile t of unit u into a stage of D / 64 chunks of 64 rows x 128
// bytes.  A page out of range reads as zeros (a TMA box outside its tensor)
// and is reported.
template <int D>
__device__ __forceinline__ void load_tile(const PageMap& m, const TileUnit& u, int t, const TilePages& pg,
                                          const CUtensorMap* map, uint8_t* stage, uint64_t* full,
                                          unsigned int* status) {
  int n = 0;
#pragma unroll
  for (int y = 0; y < 4; ++y) n += m.live(u, t, y) ? 1 : 0;
  mbar_arrive_expect_tx(full, static_cast<uint32_t>(n) << (m.log_box + (D == 64 ? 7 : 8)));
  const int x = (t * kStepKeys) & ((1 << m.log_page) - 1);  // row in the page; 0 for pages of up to 64 rows
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    if (!m.live(u, t, y)) continue;
    int page = pg.id[y];
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(m.n_pages)) {
      atomicOr(status, kStatusPagesBit);
      page = m.n_pages;
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_load_4d(stage + c * kStepKeys * 128 + (y << (m.log_box + 7)), map, full, c * 64, x, u.h, page);
  }
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

// A piece's row goes to the workspace; the warp whose 32 rows complete their
// unit joins the pieces in order, so the result does not depend on which it
// is, with weights 2^(lse_c - max).
template <int D, bool O_BF16>
__device__ __forceinline__ void store_piece(const TileUnit& u, int quad, int lane, const float (&ov)[D], float lse2,
                                            float* part, int* counters, void* o, float* lse, int T, int H) {
  const int a = quad * 32 + lane;
  constexpr size_t kPart = kTileQueries * (D + 1);
  {
    float* mine = part + plan_place(static_cast<int>(blockIdx.x), u.index) * kPart;
    float4* po = reinterpret_cast<float4*>(mine + a * D);
#pragma unroll
    for (int c = 0; c < D / 4; ++c) __stcg(po + c, make_float4(ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]));
    __stcg(mine + kTileQueries * D + a, lse2);
  }
  __threadfence();  // the piece's rows are visible before it is counted
  __syncwarp();
  int arrived = 0;
  if (lane == 0) arrived = atomicAdd(counters + u.first * 4 + quad, 1);
  if (__shfl_sync(0xffffffffu, arrived, 0) != u.pieces - 1) return;
  __threadfence();
  float top = -INFINITY;
  for (int y = 0; y < u.pieces; ++y)
    top = fmaxf(top, __ldcg(part + plan_place(u.first + y, y) * kPart + kTileQueries * D + a));
  const float eff = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int y = 0; y < u.pieces; ++y)
    sum += ex2(__ldcg(part + plan_place(u.first + y, y) * kPart + kTileQueries * D + a) - eff);
  const float inv = top == -INFINITY ? 0.f : 1.f / sum;
  if (a >= u.nq) return;
  const size_t at = (static_cast<size_t>(u.row0 + a) * H + u.h) * D;
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {
    float acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0.f;
    for (int y = 0; y < u.pieces; ++y) {
      const float* from = part + plan_place(u.first + y, y) * kPart;
      const float w = ex2(__ldcg(from + kTileQueries * D + a) - eff);
      const float4* src = reinterpret_cast<const float4*>(from + a * D + c0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 x = __ldcg(src + e);
        acc[4 * e] = fmaf(w, x.x, acc[4 * e]);
        acc[4 * e + 1] = fmaf(w, x.y, acc[4 * e + 1]);
        acc[4 * e + 2] = fmaf(w, x.z, acc[4 * e + 2]);
        acc[4 * e + 3] = fmaf(w, x.w, acc[4 * e + 3]);
      }
    }
    if (O_BF16) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o) + at + c0);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dst[e] = make_uint4(
            pack_bf16x2(acc[8 * e] * inv, acc[8 * e + 1] * inv), pack_bf16x2(acc[8 * e + 2] * inv, acc[8 * e + 3] * inv),
            pack_bf16x2(acc[8 * e + 4] * inv, acc[8 * e + 5] * inv),
            pack_bf16x2(acc[8 * e + 6] * inv, acc[8 * e + 7] * inv));
    } else {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(o) + at + c0);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dst[e] = make_float4(acc[4 * e] * inv, acc[4 * e + 1] * inv, acc[4 * e + 2] * inv, acc[4 * e + 3] * inv);
    }
  }
  if (lse != nullptr)
    lse[static_cast<size_t>(u.h) * T + u.row0 + a] =
        top == -INFINITY ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
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
  int* counters;
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

cudaError_t launch_paged_tc64(const TileMaps& m, const TileParams& p, bool o_bf16, int sms, cudaStream_t stream);
cudaError_t launch_paged_tc128(const TileMaps& m, const TileParams& p, bool o_bf16, int sms, cudaStream_t stream);

}  // namespace txl
