// How the bf16 paged attention divides its work, from the lengths on the
// device.
//
// A unit is a (sequence, head, query tile) with nks key steps of its visible
// rows.  It costs kUnit + kStep nks; the units stand in order of sequence,
// head, tile, and the line of their costs (length S) is cut into `ctas` equal
// ranges, one per CTA: CTA c has [c S / ctas, (c+1) S / ctas).  A key step
// belongs to the CTA in whose range its last cost position lies, so a unit
// that a cut falls into becomes pieces on consecutive CTAs; their results are
// joined through the workspace.  Every CTA then has the same work whatever
// the lengths are, few long sequences included, and a CTA has at most two
// pieces that are not whole units.
//
// Decoding units (up to kDecodeRows queries) and tiles of 128 queries are
// divided apart, each kind over the CTAs of its own kernel.
#pragma once

#include <cuda_runtime.h>

#include "pages.h"

namespace txl {

constexpr int kDecodeRows = 4;  // sequences with up to this many new tokens go to the decode kernel
constexpr int kMaxSms = 160;    // CTAs that the workspace has room for, per SM slot of a kernel
constexpr int kDecodePerSm = 2;
constexpr int kTileQueries = 128;

// One sequence of a kind, in the order of the call.
struct __align__(16) PlanSeq {
  long long pre;  // cost of the sequences before it
  int tok0, n, slot, start, rows, pad;
};
static_assert(sizeof(PlanSeq) == 32, "two 16-byte loads");

// One kind's division.
struct __align__(16) PlanHead {
  long long total;  // S
  int count;        // sequences
  int ctas;         // CTAs with work (0: none)
};

template <int W, int U>
struct PlanCost {
  static constexpr int kStep = W;  // cost of a key step
  static constexpr int kUnit = U;  // cost of a unit besides its steps
};
// In half key steps: what a unit costs besides its steps is set by its
// queries' load and its epilogue.
using DecodeCost = PlanCost<2, 3>;
using TileCost = PlanCost<2, 3>;

// Key steps of `BK` rows from the first live row to row x (page rows counted
// from the slot's first page); at least one.
__host__ __device__ __forceinline__ int plan_steps(int start, int x, int BK) {
  return x < start ? 1 : x / BK - start / BK + 1;
}

// The CTA whose range of the line holds position x.
__host__ __device__ __forceinline__ int plan_owner(long long x, long long total, int ctas) {
  return static_cast<int>(((x + 1) * ctas - 1) / total);
}

// A piece of a unit: key steps [t0, t0 + nks) counted from the slot's first
// page; of `pieces` the `index`-th, `first` the CTA that has the 0-th.
struct Piece {
  int t0, nks, first, index, pieces;
};

// CTA c's (range [lo, hi)) piece of the unit at cost position a with `steps`
// key steps from step `base`; nks = 0: none of its steps are c's.
template <typename Cost>
__host__ __device__ __forceinline__ Piece plan_piece(long long a, int steps, int base, int c, long long lo,
                                                     long long hi, long long total, int ctas) {
  const long long s0 = a + Cost::kUnit;
  long long from = lo < s0 ? 0 : (lo - s0) / Cost::kStep;
  long long to = hi < s0 ? 0 : (hi - s0) / Cost::kStep;
  if (from > steps) from = steps;
  if (to > steps) to = steps;
  Piece p;
  p.t0 = base + static_cast<int>(from);
  p.nks = static_cast<int>(to - from);
  p.first = c;
  p.index = 0;
  p.pieces = 1;
  if (p.nks > 0 && p.nks < steps) {
    p.first = plan_owner(s0 + Cost::kStep - 1, total, ctas);
    p.index = c - p.first;
    p.pieces = plan_owner(s0 + static_cast<long long>(Cost::kStep) * steps - 1, total, ctas) - p.first + 1;
  }
  return p;
}

// Where a partial result of CTA c lies: a piece that starts its unit and one
// that continues an earlier CTA's have a place each.
__host__ __device__ __forceinline__ int plan_place(int c, int index) { return 2 * c + (index == 0 ? 1 : 0); }

// The plan's data as a kernel reads it: from L2, since a kernel that overlaps
// the one ahead of it on the stream may find older lines in L1.
__host__ __device__ __forceinline__ PlanSeq plan_load(const PlanSeq* p) {
#ifdef __CUDA_ARCH__
  union {
    int4 v[2];
    PlanSeq s;
  } u;
  u.v[0] = __ldcg(reinterpret_cast<const int4*>(p));
  u.v[1] = __ldcg(reinterpret_cast<const int4*>(p) + 1);
  return u.s;
#else
  return *p;
#endif
}
__host__ __device__ __forceinline__ int plan_load(const int* p) {
#ifdef __CUDA_ARCH__
  return __ldcg(p);
#else
  return *p;
#endif
}
#ifdef __CUDACC__
__device__ __forceinline__ PlanHead plan_load(const PlanHead* p) {
  union {
    int4 v;
    PlanHead h;
  } u;
  u.v = __ldcg(reinterpret_cast<const int4*>(p));
  return u.h;
}
#endif

// A walk over the units that CTA c has steps of.  Every role of a CTA walks
// by itself.  BK: rows of a key step; TILE: queries of a unit (0: the unit
// has all of the sequence's).
template <typename Cost, int BK, int TILE>
struct PlanWalk {
  const PlanSeq* seqs;
  PlanHead head;
  int H, c, i, h, qt;
  PlanSeq s;
  long long a, lo, hi;  // cost position of the unit, the CTA's range
  Piece p;

  __host__ __device__ __forceinline__ int steps_of(int tile) const {
    const int m = s.start + s.rows - s.n;  // page row of query 0
    const int last = TILE == 0 ? s.n - 1 : (tile * TILE + TILE < s.n ? tile * TILE + TILE : s.n) - 1;
    return plan_steps(s.start, m + last, BK);
  }
  __host__ __device__ __forceinline__ int tiles() const { return TILE == 0 ? 1 : (s.n + TILE - 1) / TILE; }
  __host__ __device__ __forceinline__ long long cost_of(int tile) const {
    return Cost::kUnit + static_cast<long long>(Cost::kStep) * steps_of(tile);
  }

  __host__ __device__ __forceinline__ long long cost_of_head() const {
    long long per = 0;
    for (int y = 0; y < tiles(); ++y) per += cost_of(y);
    return per;
  }

  // The CTA's first unit with a step in its range; false: none.
  __host__ __device__ __forceinline__ bool begin(const PlanSeq* list, const PlanHead& hd, const int* starts, int heads, int cta) {
    seqs = list;
    head = hd;
    H = heads;
    c = cta;
    if (c >= head.ctas) return false;
    i = plan_load(starts + c);
    s = plan_load(seqs + i);
    lo = c * head.total / head.ctas;
    hi = (c + 1LL) * head.total / head.ctas;
    const long long per = cost_of_head();
    h = static_cast<int>((lo - s.pre) / per);
    a = s.pre + h * per;
    qt = 0;
    while (a + cost_of(qt) <= lo) a += cost_of(qt++);
    return settle();
  }
  __host__ __device__ __forceinline__ bool next() {
    step_unit();
    return settle();
  }

 private:
  __host__ __device__ __forceinline__ void step_unit() {
    a += cost_of(qt);
    if (++qt < tiles()) return;
    qt = 0;
    if (++h < H) return;
    h = 0;
    if (++i < head.count) s = plan_load(seqs + i);
  }
  __host__ __device__ __forceinline__ bool settle() {
    for (; i < head.count && a < hi; step_unit()) {
      p = plan_piece<Cost>(a, steps_of(qt), s.start / BK, c, lo, hi, head.total, head.ctas);
      if (p.nks > 0) return true;
    }
    return false;
  }
};

using DecodeWalk64 = PlanWalk<DecodeCost, 64, 0>;  // D = 64
using DecodeWalk32 = PlanWalk<DecodeCost, 32, 0>;  // D = 128
using TileWalk = PlanWalk<TileCost, 64, kTileQueries>;

// CTAs that share a line of length `total`: a CTA's range holds at least two
// key steps, so every CTA between a unit's first and last has one of its
// steps.
template <typename Cost>
__host__ __device__ __forceinline__ int plan_ctas(long long total, int count, int most) {
  const long long want = total / (2 * Cost::kStep);
  return count == 0 ? 0 : (want >= most ? most : (want < 1 ? 1 : static_cast<int>(want)));
}

// A tile unit that a cut divides, noted by the CTA that has its first piece.
struct TileCut {
  int row0, nq, h, pieces;  // pieces 0: none
};

// The workspace of a call.
struct PlanSpace {
  PlanHead* heads;    // [2] decode, tiles
  int* starts[2];     // [CTAs of the kind] first sequence of each CTA
  PlanSeq* seqs[2];   // [n]
  int* counters;      // [decode CTAs][4] pieces of the unit that the CTA starts which have arrived
  TileCut* cuts;      // [tile CTAs]
  float* part[2];     // [2 CTAs] partial results
};
constexpr int kDecodeCtas = kDecodePerSm * kMaxSms, kTileCtas = kMaxSms;

// Floats of one partial result: o and (m, l), or o and lse, of each row.
constexpr long long decode_part(int D) { return kDecodeRows * (D + 2LL); }
constexpr long long tile_part(int D) { return kTileQueries * (D + 1LL); }

inline size_t plan_space(void* base, int n, int T, int D, PlanSpace* out) {
  char* p = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = p + at;
    at += (bytes + 255) / 256 * 256;
    return q;
  };
  const bool tiles = T > kDecodeRows;  // else no sequence can have a tile
  PlanSpace s{};
  s.heads = reinterpret_cast<PlanHead*>(take(2 * sizeof(PlanHead)));
  for (int k = 0; k < 2; ++k) {
    const int ctas = k == 0 ? kDecodeCtas : kTileCtas;
    if (k == 1 && !tiles) break;
    s.starts[k] = reinterpret_cast<int*>(take(ctas * sizeof(int)));
    s.seqs[k] = reinterpret_cast<PlanSeq*>(take(static_cast<size_t>(n) * sizeof(PlanSeq)));
    if (k == 0)
      s.counters = reinterpret_cast<int*>(take(ctas * 4 * sizeof(int)));
    else
      s.cuts = reinterpret_cast<TileCut*>(take(ctas * sizeof(TileCut)));
    s.part[k] = reinterpret_cast<float*>(
        take(2 * static_cast<size_t>(ctas) * (k == 0 ? decode_part(D) : tile_part(D)) * sizeof(float)));
  }
  if (out != nullptr) *out = s;
  return at;
}

cudaError_t launch_paged_plan(const PagedAttn& a, const PlanSpace& s, int decode_bk, int sms, unsigned int* status,
                              cudaStream_t stream);
cudaError_t launch_paged_join(const PagedAttn& a, const PlanSpace& s, int sms, cudaStream_t stream);
// behind_tiles: launched behind the tile kernel, not behind the plan.
cudaError_t launch_paged_decode(const PagedAttn& a, const PlanSpace& s, int sms, bool behind_tiles, const WaitCtl& wc,
                                cudaStream_t stream);
// The pieces of every CTA of a kind (0: decode at head dimension D, 1: tiles) for n valid sequences, as rows (cta,
// sequence, head, tile, t0, nks, first, index, pieces, place); host only.  Returns their number, -1 if cap is short.
int paged_pieces(int kind, int D, int H, int n, const int* start, const int* rows, const int* fresh, int ctas, int* out,
                 int cap);
int paged_sms();

}  // namespace txl
