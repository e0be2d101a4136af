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
// (plan_begin: all of its threads sum the sequences' costs); then a warp finds
// its units, 32 at a time (plan_batch).  That takes about 4 us of the 104 that 22
// sequences of 512 tokens over 512 rows take (8 heads), half of it two trips to
// L2, where a kernel that made a list for all CTAs took 5 and a launch.
//
// Three kernels divide their own sequences: those of up to kDecodeRows new
// tokens (bf16), those of more (bf16, tiles of 128 queries), all (fp32, tiles
// of 16 queries).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "pages.h"

namespace txl {

// Sequences with up to this many new tokens go to the decode kernel, whose eight
// columns hold four queries in two parts.  (1 to 4 tokens there and in tiles: 64
// sequences over 300 to 4500 rows, 16 heads of 64, 97 to 104 us and 286; 48 over
// 1600 to 8100 rows, 8 heads of 128, 157 to 170 and 292; 256 over 64 rows, 8 heads
// of 64, 27 to 31 and 74.)
constexpr int kDecodeRows = 4;
constexpr int kMaxSms = 160;    // the workspace has room for the CTAs of so many SMs
constexpr int kDecodePerSm = 2, kSimtPerSm = 3;
constexpr int kTileQueries = 128, kSimtQueries = 16;

// One sequence.
struct __align__(16) PlanSeq {
  long long pre;  // cost of the sequences before it
  long long per;  // cost of one head
  int tok0, n, slot, start, rows;
};

template <int W, int U, int L>
struct PlanCost {
  static constexpr int kStep = W;   // cost of a key step
  static constexpr int kUnit = U;   // cost of a unit besides its steps
  static constexpr int kLeast = L;  // key steps that a CTA's range holds at least
};
// In half key steps: what a unit costs besides its steps is set by its
// queries' load and its epilogue.  (Measured on ragged batches: tiles 103.6 us at
// 5, 105.4 at 7, 109.1 at 11; 8 sequences of 768 tokens, D = 128, 111.3, 110.8 and
// 111.1; fp32 27.0 at 1, 24.9 at 3, 28.1 at 4; decode within 0.5% from 2 to 6.
// Small calls are split as far as it pays: a token over 512 rows 9.0 us with two
// steps a range at least, 9.5 with one; 4 sequences of up to 56 tokens in fp32,
// whose steps are long, 12.3 and 10.8.)
using DecodeCost = PlanCost<2, 4, 2>;
using TileCost = PlanCost<2, 7, 2>;
using SimtCost = PlanCost<2, 3, 1>;

// Key steps of `BK` rows from the first live row to row x (page rows counted
// from the slot's first page); at least one.
__host__ __device__ __forceinline__ int plan_steps(int start, int x, int BK) {
  return x < start ? 1 : x / BK - start / BK + 1;
}

// The line of costs: its length and how the CTAs share it.  (What a CTA does
// at its head is a chain of dependent instructions, so one division by ctas is
// all there is, in 32 bits where the length allows.)
struct PlanLine {
  long long total, each;  // each: floor(total / ctas)
  int ctas, rest;
  float rate, inv;        // ctas / total, 1 / ctas
};
__host__ __device__ __forceinline__ PlanLine plan_line(long long total, int ctas) {
  PlanLine l{total, 0, ctas, 0, 0.f, 0.f};
  if (ctas > 0) {
    l.each = total >> 32 ? total / ctas : static_cast<uint32_t>(total) / static_cast<uint32_t>(ctas);
    l.rest = static_cast<int>(total - l.each * ctas);
    l.inv = 1.f / static_cast<float>(ctas);
    l.rate = static_cast<float>(ctas) / static_cast<float>(total);
  }
  return l;
}

// Where CTA c's range begins: floor(c total / ctas) = c each + floor(c rest / ctas).
__host__ __device__ __forceinline__ long long plan_cut(int c, const PlanLine& l) {
  const int x = c * l.rest;  // c, rest < ctas < 2^10: exact in fp32, the estimate off by one at most
  int q = static_cast<int>(static_cast<float>(x) * l.inv);
  const int r = x - q * l.ctas;
  q += (r >= l.ctas) - (r < 0);
  return c * l.each + q;
}

// The CTA whose range of the line holds position x: the largest c with
// plan_cut(c) <= x.  The estimate is off by one at most.
__host__ __device__ __forceinline__ int plan_owner(long long x, const PlanLine& l) {
  int c = static_cast<int>(static_cast<float>(x) * l.rate);
  c = c < l.ctas ? c : l.ctas - 1;
  const bool less = plan_cut(c, l) > x, more = c + 1 < l.ctas && plan_cut(c + 1, l) <= x;
  return c + more - less;
}

// CTAs that share a line of length `total`: a CTA's range is kLeast key steps
// long at least, so every CTA between a unit's first and last has one of its
// steps.
template <typename Cost>
__host__ __device__ __forceinline__ int plan_ctas(long long total, int most) {
  static_assert(Cost::kStep == 2 && (Cost::kLeast == 1 || Cost::kLeast == 2), "a shift");
  const long long want = total >> Cost::kLeast;
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
                                                     long long hi, const PlanLine& line) {
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
    p.first = plan_owner(s0 + Cost::kStep - 1, line);
    p.index = c - p.first;
    p.pieces = plan_owner(s0 + static_cast<long long>(Cost::kStep) * steps - 1, line) - p.first + 1;
  }
  return p;
}

// Where a partial result of CTA c lies: a piece that starts its unit and one
// that continues an earlier CTA's have a place each.
__host__ __device__ __forceinline__ int plan_place(int c, int index) { return 2 * c + (index == 0 ? 1 : 0); }

// A unit: entry of the list at hand, head, tile.
struct PlanAt {
  int i, h, qt;
};

// The units of a kernel.  BK: rows of a key step; TILE: queries of a unit (0:
// the unit has all of the sequence's); sequences of kLo to kHi new tokens are
// the kernel's.  Everything is found in closed form, so that the lanes of a
// warp find a CTA's next 32 units at once (plan_batch).  (One after the other,
// each cost the warp that loads the tiles about 3000 cycles: 600 dependent
// instructions, the first time fetched as they run.)
template <typename C, int BK, int TILE, int LO, int HI>
struct PlanUnits {
  using Cost = C;
  static constexpr int kLo = LO, kHi = HI;

  static __host__ __device__ __forceinline__ int tiles_of(const PlanSeq& s) {
    return TILE == 0 ? 1 : (s.n + TILE - 1) / (TILE == 0 ? 1 : TILE);
  }
  static __host__ __device__ __forceinline__ int steps_of(const PlanSeq& s, int tile) {
    const int m = s.start + s.rows - s.n;  // page row of query 0
    const int last = TILE == 0 ? s.n - 1 : (tile * TILE + TILE < s.n ? tile * TILE + TILE : s.n) - 1;
    return plan_steps(s.start, m + last, BK);
  }
  // A sequence's units of one head before tile `to`: kUnit each, and the steps.
  // Tile y of those before the last ends at row m + y TILE + TILE - 1 = x, its
  // last key step is floor(x / BK).
  static __host__ __device__ __forceinline__ long long cost_before(const PlanSeq& s, int to) {
    const int tiles = tiles_of(s), whole = to < tiles ? to : tiles - 1;
    long long steps = to == tiles ? steps_of(s, tiles - 1) : 0;
    if (TILE != 0 && whole > 0) {
      const int m = s.start + s.rows - s.n;
      // the first y0 tiles end before the first live row (rows < n): a step each
      int y0 = m < s.start ? (s.start - m) / (TILE == 0 ? 1 : TILE) : 0;
      y0 = y0 < whole ? y0 : whole;
      const int k = whole - y0;
      steps += y0;
      if (k > 0) {
        const uint32_t first = m + y0 * TILE + TILE - 1;  // no less than start
        const int base = static_cast<int>(static_cast<uint32_t>(s.start) / BK) - 1;
        if (TILE >= BK) {  // floor(x / BK) grows by TILE / BK a tile
          constexpr int kBy = TILE / BK;
          steps += static_cast<long long>(k) * (static_cast<int>(first / BK) - base) +
                   kBy * (static_cast<long long>(k) * (k - 1) >> 1);
        } else {  // floor(x / BK) = floor((b + y) / 2)
          static_assert(TILE == 0 || TILE >= BK || 2 * TILE == BK, "half a key step a tile");
          auto halves = [](int z) { return z < 1 ? 0 : static_cast<long long>(z - 1) * (z - 1) >> 2; };  // sum of floor(j / 2), j < z
          const int b = first / (TILE == 0 ? 1 : TILE);
          steps += halves(b + k) - halves(b) - static_cast<long long>(k) * base;
        }
      }
    }
    return static_cast<long long>(Cost::kUnit) * to + Cost::kStep * steps;
  }
  static __host__ __device__ __forceinline__ long long cost_of_head(const PlanSeq& s) {
    return cost_before(s, tiles_of(s));
  }

  // The unit of sequence s (list[0]) that position x of the line lies in.
  static __host__ __device__ __forceinline__ PlanAt place(const PlanSeq& s, long long x) {
    const long long per = s.per, past = x - s.pre;
#ifdef __CUDA_ARCH__
    const float ratio = __fdividef(static_cast<float>(past), static_cast<float>(per));
#else
    const float ratio = static_cast<float>(past) / static_cast<float>(per);
#endif
    PlanAt at{0, static_cast<int>(ratio), 0};  // off by one at most: h < 2^20
    at.h -= at.h > 0 && at.h * per > past;
    at.h += (at.h + 1) * per <= past;
    if (TILE != 0) {
      const long long in = past - at.h * per;
      int hi = tiles_of(s);  // the largest qt with cost_before(qt) <= in
      while (at.qt + 1 < hi) {
        const int mid = (at.qt + hi) >> 1;
        if (cost_before(s, mid) <= in)
          at.qt = mid;
        else
          hi = mid;
      }
    }
    return at;
  }
  // The r-th unit (r < 32) behind `from` of the `count` entries of `list` (n = 0: not
  // the kernel's); false: there is none.
  static __host__ __device__ __forceinline__ bool find(const PlanSeq* list, int count, int H, PlanAt from, int r,
                                                       PlanAt* to) {
    for (; from.i < count; ++from.i) {
      if (list[from.i].n == 0) continue;  // from.h, from.qt are 0 here
      const int tiles = tiles_of(list[from.i]), x = from.qt + r;
      const int dh = static_cast<uint32_t>(x) / static_cast<uint32_t>(tiles);
      if (from.h + dh < H) {
        *to = PlanAt{from.i, from.h + dh, x - dh * tiles};
        return true;
      }
      r -= (H - from.h) * tiles - from.qt;  // no more than r
      from.h = from.qt = 0;
    }
    return false;
  }
  // CTA c's (range [lo, hi)) piece of a unit; nks = 0: none of its steps are c's.
  static __host__ __device__ __forceinline__ Piece piece(const PlanSeq& s, PlanAt at, int c, long long lo, long long hi,
                                                         const PlanLine& line) {
    const long long a = s.pre + at.h * s.per + (TILE == 0 ? 0 : cost_before(s, at.qt));
    if (a >= hi) return Piece{0, 0, 0, 0, 0};
    return plan_piece<Cost>(a, steps_of(s, at.qt), s.start / BK, c, lo, hi, line);
  }
};
using DecodeUnits64 = PlanUnits<DecodeCost, 64, 0, 1, kDecodeRows>;  // D = 64
using DecodeUnits32 = PlanUnits<DecodeCost, 32, 0, 1, kDecodeRows>;  // D = 128
using TileUnits = PlanUnits<TileCost, 64, kTileQueries, kDecodeRows + 1, 0x7fffffff>;
using SimtUnits = PlanUnits<SimtCost, 32, kSimtQueries, 1, 0x7fffffff>;

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
  PlanLine line;
  long long pre;    // cost of the entries before `raw`
  int raw;          // the next entry to read
  int from, count;  // entry that the CTA's range starts in; entries at hand in `seqs`
  PlanAt next;      // the unit to find next, in `seqs`
  union {
    long long sums[2][16];  // plan_begin: warps' sums (up to 16 warps)
    PlanSeq seqs[32];       // behind its next to last barrier
  };
};

// All threads of the CTA (a multiple of 32, up to 512): S, the CTAs that share
// it, the entry that this CTA's range starts in and, of lists that the CTA
// reads in one go, the entries from there on.  Ends with a barrier.
template <typename Units>
__device__ __forceinline__ void plan_begin(const PlanArgs& p, int most, PlanState* st) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int c = static_cast<int>(blockIdx.x);
  bool bad = false;
  PlanSeq s{};
  PlanLine line{};
  long long upto = 0, lo = -1, mine = 0;  // upto: cost of the entries so far; lo: the range's start, once known
  // Blocks of nt entries: the total, then, if there are several, again up to
  // the one that the range starts in.
#pragma unroll 1
  for (int base = 0, turn = 0;; turn ^= 1) {
    s.n = 0;
    if (base + tid < p.n) s = plan_read(p, base + tid, Units::kLo, Units::kHi, &bad);
    if (s.n > 0) s.per = Units::cost_of_head(s);
    mine = s.n > 0 ? s.per * p.H : 0;
    const long long x = warp_scan(mine);
    if (lane == 31) st->sums[turn][warp] = x;
    __syncthreads();
    long long before = upto + x - mine;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      const long long y = w < nw ? st->sums[turn][w] : 0;
      before += w < warp ? y : 0;
      upto += y;
    }
    base += nt;
    if (lo < 0 && base >= p.n) {
      line = plan_line(upto, plan_ctas<typename Units::Cost>(upto, most));
      if (c >= line.ctas) break;
      lo = plan_cut(c, line);
      if (p.n > nt) {
        base = 0;
        upto = 0;
        continue;
      }
    }
    if (lo >= 0) {
      if (mine > 0 && before <= lo && lo < before + mine) {
        st->from = st->raw = base - nt + tid;
        st->pre = before;
      }
      s.pre = before;
      if (upto > lo) break;
    }
  }
  if (bad && c == 0) atomicOr(p.status, kStatusPagesBit);
  if (tid == 0) {
    st->line = line;
    st->count = 0;
  }
  __syncthreads();
  if (p.n > nt || c >= line.ctas) return;
  // (Read again by the warp that finds the units, they cost 2 us of every call.)
  const int from = st->from, k = tid - from, count = min(32, p.n - from);
  if (k >= 0 && k < count) {
    st->seqs[k] = s;
    if (k == count - 1) {
      st->raw = from + count;
      st->pre = s.pre + mine;
      st->count = count;
    }
  }
  __syncthreads();
}

// One warp: the next entries, up to 32 (0: there are none), from entry st->raw
// on, into st->seqs.
template <typename Units>
__device__ __forceinline__ int plan_fill(const PlanArgs& p, PlanState* st) {
  const int lane = threadIdx.x & 31;
  const int raw = st->raw, count = max(0, min(32, p.n - raw));
  const long long pre = st->pre;
  __syncwarp();
  PlanSeq s{};
  bool bad = false;
  if (lane < count) s = plan_read(p, raw + lane, Units::kLo, Units::kHi, &bad);
  if (s.n > 0) s.per = Units::cost_of_head(s);
  const long long cost = s.n > 0 ? s.per * p.H : 0;
  const long long upto = warp_scan(cost);
  s.pre = pre + upto - cost;
  if (lane < count) st->seqs[lane] = s;
  if (lane == 31) {
    st->raw = raw + count;
    st->pre = pre + upto;
  }
  __syncwarp();
  return count;
}

// A unit that a lane found.
struct PlanFound {
  PlanSeq s;
  int h, qt;
  Piece p;
};

// One warp, behind plan_begin: the CTA's next units, up to 32 (`first`: its
// first ones), lane by lane; their number, 0 only where *last.  *last: there
// are no more behind them.
template <typename Units>
__device__ __forceinline__ int plan_batch(const PlanArgs& p, PlanState* st, bool first, PlanFound* f, bool* last) {
  const int lane = threadIdx.x & 31, c = static_cast<int>(blockIdx.x);
  const PlanLine line = st->line;
  *last = true;
  if (c >= line.ctas) return 0;
  const long long lo = plan_cut(c, line), hi = plan_cut(c + 1, line);
  PlanAt from = st->next;
  int count = st->count, found = 0;
  bool fresh = first;
#pragma unroll 1
  for (;;) {
    if (count == 0 && (count = plan_fill<Units>(p, st)) == 0) {
      *last = true;
      return 0;
    }
    if (fresh) from = Units::place(st->seqs[0], lo);
    fresh = false;
    PlanAt at{};
    const bool any = Units::find(st->seqs, count, p.H, from, lane, &at);
    f->p.nks = 0;
    if (any) {
      f->s = st->seqs[at.i];
      f->h = at.h;
      f->qt = at.qt;
      f->p = Units::piece(f->s, at, c, lo, hi, line);
    }
    // The lanes with a unit come first: those behind the range's end, or the
    // list's, have none.
    found = __popc(__ballot_sync(0xffffffffu, f->p.nks > 0));
    *last = __any_sync(0xffffffffu, any && f->p.nks == 0);
    __syncwarp();
    if (!__all_sync(0xffffffffu, any) && !*last) {  // the list is used up
      *last = st->raw >= p.n;
      count = 0;
      from = PlanAt{0, 0, 0};
    } else {
      from.i = __shfl_sync(0xffffffffu, at.i, 31);
      from.h = __shfl_sync(0xffffffffu, at.h, 31);
      from.qt = __shfl_sync(0xffffffffu, at.qt, 31) + 1;  // past the head's last tile: find() goes on
    }
    if (found > 0 || *last) break;
  }
  if (lane == 0) {
    st->next = from;
    st->count = count;
  }
  __syncwarp();
  return found;
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
// ahead_of_tiles: the tile kernel follows.
cudaError_t launch_paged_decode(const PagedAttn& a, const PlanSpace& s, int sms, bool ahead_of_tiles, const WaitCtl& wc,
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
