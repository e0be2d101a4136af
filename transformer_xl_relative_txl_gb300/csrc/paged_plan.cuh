// How the paged attention divides its work, from the lengths on the device.
//
// A unit is a (sequence, head, query tile) with nks key steps of its visible
// rows.  It costs kUnit + kStep nks; the units stand in order of sequence,
// head, tile, and the line of their costs (length S) is cut into `ctas` equal
// ranges, one per CTA: CTA c has [c S / ctas, (c+1) S / ctas).  A key step
// belongs to the CTA in whose range its last cost position lies, so a unit
// that a cut falls into becomes pieces on consecutive CTAs, which the kernel
// of paged_join.cu joins.  Every CTA then has the same work whatever the
// lengths are, few long sequences included, and a CTA has at most two pieces
// that are not whole units.
//
// Each CTA finds S and the start of its own range by itself, at its head
// (plan_begin: all of its threads sum the sequences' costs), and then reads the
// sequences of its range 32 at a time (plan_fill).  That takes about 2 us where
// a kernel that made a list for all CTAs took 5 and a launch.
//
// Three kernels divide their own sequences: those of up to kDecodeRows new
// tokens (bf16), those of more (bf16, tiles of 128 queries), all (fp32, tiles
// of 16 queries).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "pages.h"

namespace txl {

constexpr int kDecodeRows = 4;  // sequences with up to this many new tokens go to the decode kernel
constexpr int kMaxSms = 160;    // the workspace has room for the CTAs of so many SMs
constexpr int kDecodePerSm = 2, kSimtPerSm = 4;
constexpr int kTileQueries = 128, kSimtQueries = 16;

// One sequence.
struct __align__(16) PlanSeq {
  long long pre;  // cost of the sequences before it
  int tok0, n, slot, start, rows, index;
};

template <int W, int U>
struct PlanCost {
  static constexpr int kStep = W;  // cost of a key step
  static constexpr int kUnit = U;  // cost of a unit besides its steps
};
// In half key steps: what a unit costs besides its steps is set by its
// queries' load and its epilogue.
using DecodeCost = PlanCost<2, 3>;
using TileCost = PlanCost<2, 5>;
using SimtCost = PlanCost<2, 1>;

// Key steps of `BK` rows from the first live row to row x (page rows counted
// from the slot's first page); at least one.
__host__ __device__ __forceinline__ int plan_steps(int start, int x, int BK) {
  return x < start ? 1 : x / BK - start / BK + 1;
}

// Where CTA c's range begins: floor(c total / ctas).  (A 64-bit division takes
// over 100 instructions; nearly every line is shorter than 2^31.)
__host__ __device__ __forceinline__ long long plan_cut(int c, long long total, int ctas) {
  if (total >> 31) return c * total / ctas;
  const uint32_t n = static_cast<uint32_t>(ctas), q = static_cast<uint32_t>(total) / n;
  const uint32_t rest = static_cast<uint32_t>(total) - q * n;
  return static_cast<long long>(c) * q + static_cast<uint32_t>(c) * rest / n;  // c, rest < ctas < 2^16
}

// The CTA whose range of the line holds position x: the largest c with
// plan_cut(c) <= x.  The estimate is off by one at most (ctas < 2^16).
__host__ __device__ __forceinline__ int plan_owner(long long x, long long total, int ctas) {
  int c = static_cast<int>(static_cast<float>(x) / static_cast<float>(total) * static_cast<float>(ctas));
  if (c >= ctas) c = ctas - 1;
  while (c > 0 && plan_cut(c, total, ctas) > x) --c;
  while (c + 1 < ctas && plan_cut(c + 1, total, ctas) <= x) ++c;
  return c;
}

// CTAs that share a line of length `total`: a CTA's range holds at least two
// key steps, so every CTA between a unit's first and last has one of its
// steps.
template <typename Cost>
__host__ __device__ __forceinline__ int plan_ctas(long long total, int most) {
  static_assert(Cost::kStep == 2, "a shift");
  const long long want = total >> 2;
  return total == 0 ? 0 : (want >= most ? most : (want < 1 ? 1 : static_cast<int>(want)));
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
  static_assert(Cost::kStep == 2, "shifts");
  long long from = lo < s0 ? 0 : (lo - s0) >> 1;
  long long to = hi < s0 ? 0 : (hi - s0) >> 1;
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

enum PlanStep { kPlanUnit, kPlanEnd, kPlanFill };

// A walk over the units that CTA c has steps of.  BK: rows of a key step;
// TILE: queries of a unit (0: the unit has all of the sequence's); sequences of
// kLo to kHi new tokens are the kernel's.
template <typename C, int BK, int TILE, int LO, int HI>
struct PlanWalk {
  using Cost = C;
  static constexpr int kLo = LO, kHi = HI;
  const PlanSeq* seqs;  // the sequences at hand
  int count;            // how many
  bool left;            // there are more behind them
  long long total;
  int ctas, H, c, i, h, qt;
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
  static __host__ __device__ __forceinline__ long long cost_of_seq(const PlanSeq& x, int heads) {
    PlanWalk w;
    w.s = x;
    return w.cost_of_head() * heads;
  }

  // The CTA's first unit with a step in its range; list[0] is the sequence
  // that the range starts in.
  __host__ __device__ __forceinline__ PlanStep begin(const PlanSeq* list, int n, bool more, long long length,
                                                     int n_ctas, int heads, int cta) {
    seqs = list;
    count = n;
    left = more;
    total = length;
    ctas = n_ctas;
    H = heads;
    c = cta;
    lo = plan_cut(c, total, ctas);
    hi = plan_cut(c + 1, total, ctas);
    i = 0;
    s = seqs[0];
    const long long per = cost_of_head();
    const long long past = lo - s.pre;
    h = past >> 31 ? static_cast<int>(past / per)
                   : static_cast<int>(static_cast<uint32_t>(past) /
                                      static_cast<uint32_t>(per < past + 1 ? per : past + 1));
    a = s.pre + h * per;
    qt = 0;
    while (a + cost_of(qt) <= lo) a += cost_of(qt++);
    return settle();
  }
  __host__ __device__ __forceinline__ PlanStep next() {
    step_unit();
    return settle();
  }
  // After kPlanFill: the next sequences are at hand.
  __host__ __device__ __forceinline__ PlanStep filled(int n, bool more) {
    count = n;
    left = more;
    i = 0;
    if (n > 0) s = seqs[0];
    return settle();
  }

 private:
  __host__ __device__ __forceinline__ void step_unit() {
    a += cost_of(qt);
    if (++qt < tiles()) return;
    qt = 0;
    if (++h < H) return;
    h = 0;
    if (++i < count) s = seqs[i];
  }
  __host__ __device__ __forceinline__ PlanStep settle() {
    for (;; step_unit()) {
      if (a >= hi) return kPlanEnd;
      if (i >= count) return left ? kPlanFill : kPlanEnd;
      p = plan_piece<Cost>(a, steps_of(qt), s.start / BK, c, lo, hi, total, ctas);
      if (p.nks > 0) return kPlanUnit;
    }
  }
};
using DecodeWalk64 = PlanWalk<DecodeCost, 64, 0, 1, kDecodeRows>;  // D = 64
using DecodeWalk32 = PlanWalk<DecodeCost, 32, 0, 1, kDecodeRows>;  // D = 128
using TileWalk = PlanWalk<TileCost, 64, kTileQueries, kDecodeRows + 1, 0x7fffffff>;
using SimtWalk = PlanWalk<SimtCost, 32, kSimtQueries, 1, 0x7fffffff>;

#ifdef __CUDACC__

// What a call says of its sequences.
struct PlanArgs {
  PageBook book;
  const int* slots;
  const int* cu;
  int n, T, max_new, n_r, H;
  unsigned int* status;
};

// Entry i; n = 0 where it is refused (noted in *bad) or not of lo .. hi tokens.
__device__ __forceinline__ PlanSeq plan_read(const PlanArgs& p, int i, int lo, int hi, bool* bad) {
  PlanSeq s{};
  s.index = i;
  s.tok0 = p.cu[i];
  const int n = p.cu[i + 1] - s.tok0;
  s.slot = p.slots[i];
  bool ok = s.slot >= 0 && s.slot < p.book.n_slots && n >= 0 && n <= p.max_new && s.tok0 >= 0 &&
            static_cast<long long>(s.tok0) + n <= p.T;
  if (ok) {
    s.start = p.book.start[s.slot];
    s.rows = p.book.rows[s.slot];
    ok = s.start >= 0 && s.start < p.book.page_rows && s.rows >= 0 && s.rows <= p.n_r &&
         static_cast<long long>(s.start) + s.rows <= static_cast<long long>(p.book.max_pages) * p.book.page_rows;
  }
  *bad |= !ok;
  s.n = ok && n >= lo && n <= hi ? n : 0;
  return s;
}

__device__ __forceinline__ long long warp_scan(long long x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// In shared memory: the division, this CTA's start, the sequences at hand.
struct PlanState {
  long long total, pre;  // S; cost of the entries before `raw`
  int ctas, raw;         // raw: the next entry to read
  union {
    long long sums[2][16];  // plan_begin: warps' sums (up to 16 warps)
    PlanSeq seqs[32];       // from plan_fill on
  };
};

// All threads of the CTA (a multiple of 32, up to 512): S, the CTAs that share
// it, the entry that this CTA's range starts in.  Ends with a barrier.
template <typename Walk>
__device__ __forceinline__ void plan_begin(const PlanArgs& p, int most, PlanState* st) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  bool bad = false;
  // Entries base .. base + nt - 1: cost of each and of those before it.
  int turn = 0;
  auto scan = [&](int base, long long* mine, long long* all) {
    const int i = base + tid;
    long long x = 0;
    if (i < p.n) {
      const PlanSeq s = plan_read(p, i, Walk::kLo, Walk::kHi, &bad);
      if (s.n > 0) x = Walk::cost_of_seq(s, p.H);
    }
    *mine = x;
    x = warp_scan(x);
    long long* sums = st->sums[turn ^= 1];
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = x - *mine, sum = 0;
    for (int w = 0; w < nw; ++w) {
      before += w < warp ? sums[w] : 0;
      sum += sums[w];
    }
    *all = sum;
    return before;
  };
  long long total = 0, mine = 0, all = 0, before = 0;
  for (int base = 0; base < p.n; base += nt) {
    before = scan(base, &mine, &all);
    total += all;
  }
  const int ctas = plan_ctas<typename Walk::Cost>(total, most);
  const int c = static_cast<int>(blockIdx.x);
  if (c < ctas) {
    const long long lo = plan_cut(c, total, ctas);
    long long upto = 0;
    for (int base = 0; base < p.n && upto <= lo; base += nt) {
      if (p.n > nt) before = scan(base, &mine, &all);  // else at hand
      if (mine > 0 && upto + before <= lo && lo < upto + before + mine) {
        st->raw = base + tid;
        st->pre = upto + before;
      }
      upto += all;
    }
  }
  if (bad && c == 0) atomicOr(p.status, kStatusPagesBit);
  if (tid == 0) {
    st->total = total;
    st->ctas = ctas;
  }
  __syncthreads();
}

// One warp: the kernel's next sequences, up to 32 (0: there are none), from
// entry st->raw on, into st->seqs.
template <typename Walk>
__device__ __forceinline__ int plan_fill(const PlanArgs& p, PlanState* st) {
  const int lane = threadIdx.x & 31;
  int raw = st->raw, count = 0;
  long long pre = st->pre;
  __syncwarp();
  while (count == 0 && raw < p.n) {
    PlanSeq s{};
    bool bad = false;
    if (raw + lane < p.n) s = plan_read(p, raw + lane, Walk::kLo, Walk::kHi, &bad);
    const long long cost = s.n > 0 ? Walk::cost_of_seq(s, p.H) : 0;
    const long long upto = warp_scan(cost);
    s.pre = pre + upto - cost;
    const uint32_t votes = __ballot_sync(0xffffffffu, s.n > 0);
    if (s.n > 0) st->seqs[__popc(votes & ((1u << lane) - 1))] = s;
    count = __popc(votes);
    pre += __shfl_sync(0xffffffffu, upto, 31);
    raw += 32;
  }
  if (lane == 0) {
    st->raw = raw;
    st->pre = pre;
  }
  __syncwarp();
  return count;
}

#endif  // __CUDACC__

// A unit that a cut divides, noted by the CTA that has its first piece.
struct PlanCut {
  int row0, nq, h, pieces;  // first row of q, queries, head; pieces 0: none
};

// The workspace of a call: per kernel, the cuts [CTAs] and the partial results
// [2 CTAs], each o [rows][D], normalised, then the log2-domain lse [rows].
struct PlanPart {
  PlanCut* cuts;
  float* part;
};
struct PlanSpace {
  PlanPart decode, tiles, simt;
};
constexpr int kDecodeCtas = kDecodePerSm * kMaxSms, kTileCtas = kMaxSms, kSimtCtas = kSimtPerSm * kMaxSms;

__host__ __device__ constexpr long long plan_part(int rows, int D) { return static_cast<long long>(rows) * (D + 1); }

inline size_t plan_space(void* base, int T, int D, bool bf16, PlanSpace* out) {
  char* p = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = p + at;
    at += (bytes + 255) / 256 * 256;
    return q;
  };
  auto part = [&](int ctas, int rows) {
    PlanPart x;
    x.cuts = reinterpret_cast<PlanCut*>(take(ctas * sizeof(PlanCut)));
    x.part = reinterpret_cast<float*>(take(2 * static_cast<size_t>(ctas) * plan_part(rows, D) * sizeof(float)));
    return x;
  };
  PlanSpace s{};
  if (bf16) {
    s.decode = part(kDecodeCtas, kDecodeRows);
    if (T > kDecodeRows) s.tiles = part(kTileCtas, kTileQueries);  // else no sequence can have a tile
  } else {
    s.simt = part(kSimtCtas, kSimtQueries);
  }
  if (out != nullptr) *out = s;
  return at;
}

#ifdef __CUDACC__
inline PlanArgs plan_args(const PagedAttn& a, unsigned int* status) {
  return PlanArgs{a.book, a.slots, a.cu, a.n, a.T, a.max_new, a.n_r, a.H, status};
}
#endif

// Joins the cut units of up to two kernels' parts (a part of 0 CTAs: none).
struct JoinPart {
  const PlanCut* cuts;
  const float* part;
  int ctas, rows;
};
cudaError_t launch_paged_join(const PagedAttn& a, const JoinPart& x, const JoinPart& y, cudaStream_t stream);
// behind_tiles: launched behind the tile kernel, whose end it need not wait
// for before its own.
cudaError_t launch_paged_decode(const PagedAttn& a, const PlanSpace& s, int sms, bool behind_tiles, const WaitCtl& wc,
                                cudaStream_t stream);
cudaError_t launch_paged_simt(const PagedAttn& a, const PlanSpace& s, int sms, unsigned int* status,
                              cudaStream_t stream);
// The pieces of every CTA of a kind (0: decode at head dimension D, 1: tiles,
// 2: fp32) for n valid sequences, as rows (cta, sequence, head, tile, t0, nks,
// first, index, pieces, place); host only.  Returns their number, -1 if cap is
// short.
int paged_pieces(int kind, int D, int H, int n, const int* start, const int* rows, const int* fresh, int ctas, int* out,
                 int cap);
int paged_sms();

}  // namespace txl
