// A token per row of logits: temperature, top-k, top-p, min-p, then the token
// at which the running sum of the kept weights passes a given uniform number.
//
//   w_i = exp((z_i - max z) / T)
//
// Top-k, then top-p of what it leaves, keep a prefix of the tokens by falling
// logit (equal ones by index), so each is a threshold: a value, and how many of
// the tokens that have this value.  Nothing is sorted.  The value is found by
// counts (top-k) or sums of weights (top-p) in equal bins between two logits,
// the bin that the border falls into again in bins, until it holds one value or
// few enough tokens to compare each with each.
//
// A row belongs to a cluster of up to 8 CTAs, each with a stretch of the
// vocabulary in its shared memory, so the logits are read once; what the CTAs count
// is added up over distributed shared memory.
//
// Sums decide tokens, so they are exact: a weight is a whole number of 2^-44 of
// the largest weight, cut off (right to 2^-39 of its own size before that), and
// 64-bit sums of at most 2^18 of them do not depend on their order.  In fp32, sums
// over 100000 tokens would name another token once in a hundred rows or so, and
// this chip's fp64 is far too slow for the exponentials.
//
// Bound by chains of dependent instructions: some 85 for 32 exact weights, 25 for 32
// logits put into bins, and ten or so barriers of a cluster, 1000 to 2000 cycles
// each with what is done between them.  One row of 32768 in bf16, top-k 50 of it
// and top-p: 8.7 us; 64 of 131072, top-k 100 to 300 and more: 26 us (17 MB: 0.65 TB/s);
// 128 of 50021 in fp32 by top-p, where every logit's weight counts: 57 us (0.45 TB/s),
// of 107000 cycles of a CTA 50000 for the weights, 17000 for the last look at the
// cells, 10000 for the counts, 7000 for the reading.  There the schedulers issue 41%
// of the time; twice the threads on a row take 8% less, and more elsewhere.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "pdl.cuh"
#include "tokens.h"
#include "txl_device.cuh"

namespace cg = cooperative_groups;

namespace txl {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kGroup = 32, kGroups = kBins / kGroup;  // bins that are first looked at together
constexpr int kFew = 256;        // tokens of a bin that are compared each with each
constexpr int kList = 512;       // or all down to a border of counts, that are sorted
constexpr int kCounted = 256;    // by counting
constexpr int kMaxCluster = 8;
constexpr int kTable = 512;      // steps of the powers' table
constexpr int kOne = 44;         // the largest weight is 2^kOne
constexpr int kCell = 256;       // tokens that a warp takes at once, 8 a lane
constexpr int kCells = 256;      // of a CTA's stretch, at most
constexpr int kLaneCells = kCells / 32;

// 2^(-j / kTable) in units of 2^-44, from nine square roots of a half by
// Newton's method.
struct Powers {
  unsigned long long v[kTable];
};
constexpr double newton_sqrt(double a) {
  double x = a < 1.0 ? 1.0 : a;
  for (int i = 0; i < 60; ++i) x = 0.5 * (x + a / x);
  return x;
}
constexpr Powers powers() {
  Powers p{};
  double root[9] = {};  // root[i] = 2^-(2^i / kTable)
  double r = 0.5;
  for (int i = 8; i >= 0; --i) root[i] = r = newton_sqrt(r);
  for (int j = 0; j < kTable; ++j) {
    double x = 1.0;
    for (int i = 0; i < 9; ++i)
      if (j >> i & 1) x *= root[i];
    p.v[j] = static_cast<unsigned long long>(x * static_cast<double>(1ULL << kOne) + 0.5);
  }
  return p;
}
__device__ constexpr Powers kPowers = powers();

// A row's logits and its T, times a power of two: log2(e) / T in two parts, the
// largest logit, the power.
struct Scale {
  float hi, lo, top, by;
};
// The power is 1 but for the ends of T.  A quarter where logits may be further
// apart than the largest float and still have weights.  2^40 where 1 / T may be
// over it; but for a largest logit whose own steps are 2^56 T or more, where every
// other weight is 0.  (In fp64 this alone would take a microsecond.)
__device__ __forceinline__ Scale scale_of(float temperature, float top) {
  constexpr float kHi = 1.442695041f, kLo = static_cast<float>(1.4426950408889634 - static_cast<double>(kHi));
  float by = 1.f;
  if (temperature > 0x1p100f) by = 0.25f;
  else if (temperature < 0x1p-100f && fabsf(top) < 0x1p-20f) by = 0x1p40f;
  const float t = temperature * by, hi = kHi / t;
  if (!(hi > 0.f) || hi > FLT_MAX) return Scale{fminf(hi, FLT_MAX), 0.f, top * by, by};
  return Scale{hi, (fmaf(-hi, t, kHi) + kLo) / t, top * by, by};
}

// p x in whole numbers, rounded up or down, exactly; 0 < p < 1.
__device__ __forceinline__ unsigned long long share_of(float p, unsigned long long x, bool up) {
  const uint32_t bits = __float_as_uint(p);
  const int e = max(1, static_cast<int>(bits >> 23));
  const unsigned long long m = (bits & 0x7fffffu) | (bits >> 23 != 0 ? 0x800000u : 0u);
  const int shift = 150 - e;  // p = m / 2^shift, 24 or more
  const unsigned long long hi = __umul64hi(m, x), lo = m * x;
  unsigned long long q, rest;
  if (shift < 64) {
    q = hi << (64 - shift) | lo >> shift;
    rest = lo << (64 - shift);
  } else if (shift < 128) {
    q = shift == 64 ? hi : hi >> (shift - 64);
    rest = lo | (shift == 64 ? 0ULL : hi << (128 - shift));
  } else {
    q = 0;
    rest = lo | hi;
  }
  return q + (up && rest != 0 ? 1ULL : 0ULL);
}

// exp((z - top) / T) in units of 2^-44.  With y = (top - z) log2(e) / T as the
// sum of two floats, y = k / 512 + r, the weight is 2^-(k/512), from the table,
// times 1 - q, q = 1 - 2^-r by its series in whole numbers of 2^-40: |r| <=
// 2^-10, so three terms do.  No branch, so that several run at once: one takes 250
// cycles, of which its instructions are a fifth.  Floats become whole numbers by adding a power of two
// and taking the bits: conversions run at an eighth of the rate.
__device__ __forceinline__ unsigned long long weight(float z, const Scale& c, const unsigned long long* table) {
  float d = fmaf(-z, c.by, c.top);
  const float back = d - c.top;
  float err = (c.top - (d - back)) - fmaf(z, c.by, back);  // top - z = d + err
  if (d > 3.0e38f) d = FLT_MAX, err = 0.f;
  const float y = fminf(d * c.hi, 45.f);  // from 45 on 0: the last shift
  const float y2 = fmaf(d, c.hi, -y) + fmaf(d, c.lo, err * c.hi);
  constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: one unit of its last place is 1
  const float at = fmaf(y, static_cast<float>(kTable), kWhole);
  const int k = __float_as_int(at) - __float_as_int(kWhole);
  const float f = fmaf(at - kWhole, -1.f / kTable, y);
  // r = f + y2: f in units of 2^-24, what that leaves and y2 (< 2^-17) in units of 2^-39
  constexpr float kCoarse = 0.75f, kFine = 0x1.8p-16f;
  const float coarse = f + kCoarse;
  const float fine = (f - (coarse - kCoarse)) + y2 + kFine;
  const int r = ((__float_as_int(coarse) - __float_as_int(kCoarse)) << 16) +
                ((__float_as_int(fine) - __float_as_int(kFine)) << 1);  // units of 2^-40
  const int x = __mulhi(r, 1488522236) << 1;        // r ln 2; ln 2 in units of 2^-31
  const int x2 = __mulhi(x, x) >> 9;                // x^2 / 2
  const int x3 = __mulhi(__mulhi(x2, x), 5592405);  // x^3 / 6: a third of 2^-8
  const int q = x - x2 + x3;
  const unsigned long long p = table[k & (kTable - 1)];
  const long long less = __mulhi(q << 1, static_cast<int>(p >> (kOne - 30)));  // units of 2^-39
  return (p - static_cast<unsigned long long>(less << (kOne - 39))) >> (k / kTable);
}

// A float's place in the order of floats, as a whole number.
__device__ __forceinline__ uint32_t ordered(float z) {
  const uint32_t u = __float_as_uint(z);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// What a CTA tells the others of its cluster, written into their memory ahead of
// a barrier; read there, an exchange would take a second way to and fro.
struct Found {
  int n;            // tokens of the bin
  uint32_t lo, hi;  // their ends, ordered
};
struct Kept {
  unsigned long long over;  // weights over the threshold
  int ties;                 // tokens at it
};
struct Mass {
  unsigned long long all, above;  // weights: of all tokens, of those above the window
};
struct Candidate {
  float z;
  int token;
};

struct alignas(16) Shared {
  unsigned long long table[kTable];
  alignas(16) unsigned long long bins[kBins];  // of the range at hand: sums of weights, or counts
  unsigned long long groups[kMaxCluster][kGroups];
  float top[kMaxCluster];
  uint32_t cut[kMaxCluster];
  int parts[kMaxCluster];
  Found found[kMaxCluster];
  Kept kept[kMaxCluster];
  Mass mass[kMaxCluster];
  Candidate seg[kList];  // a part for each CTA
  Candidate cand[kList];
  unsigned long long cand_w[kFew];
  unsigned long long warp_sum[kWarps];
  float warp_top[kWarps];
  uint32_t warp_cut[kWarps];
  int warp_parts[kWarps];
  unsigned long long cell_over[kCells];
  int cell_ties[kCells];
  uint32_t lo, hi;  // of a bin's tokens in this CTA
  int n;            // how many
  int bin;                           // where the border lies,
  unsigned long long above, in_bin;  // the sum ahead of it, and its own
  float value;
  unsigned long long value_above;
};
static_assert(sizeof(Shared) % 16 == 0, "the stretch behind it is read 16 bytes at a time");

// Inclusive sum over a warp.
template <typename T>
__device__ __forceinline__ T warp_scan(T x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The bins of a range of logits, largest first: linear between its ends, or by
// the floats' order where `keys` (for ranges that the linear map does not
// separate).  Either falls with z; nothing else is asked of it.
struct Range {
  float lo, hi;
  bool keys;
  int shift;
  float per, at_hi;  // bins per unit, bins of the upper end from 0
  __device__ __forceinline__ void set(float l, float h, bool k) {
    lo = l, hi = h, keys = k;
    const uint32_t span = ordered(h) - ordered(l);
    shift = max(0, 32 - __clz(span) - 10);
    per = (kBins - 1) * 0.5f / (0.5f * h - 0.5f * l);
    at_hi = h * per;
  }
  __device__ __forceinline__ bool has(float z) const { return z >= lo && z <= hi; }
  __device__ __forceinline__ int bin(float z) const {
    if (keys) return static_cast<int>((ordered(hi) - ordered(z + 0.f)) >> shift);  // (-0 is 0)
    const float x = fmaxf(fminf(fmaf(z, -per, at_hi), kBins - 1.f), 0.f);
    return __float_as_int(x + 8388608.f) & (2 * kBins - 1);
  }
  // How far a linear bin's token is behind its middle, in kOffset-ths of a bin.
  static constexpr float kOffset = 16384.f;
  __device__ __forceinline__ int offset(float z, int b) const {
    const float x = fmaf(z, -per, at_hi) - static_cast<float>(b);
    return __float2int_rn(fminf(fmaxf(x, -0.5f), 0.5f) * kOffset);
  }
  // Ends outside of which no token is in bin b (or in a later one, in an earlier).
  __device__ __forceinline__ void near(int b, float* from, float* to) const {
    const bool fine = !keys && fabsf(at_hi) < 1048576.f && fabsf(lo * per) < 1048576.f && per > 0x1p-100f;
    *from = fine ? fmaxf(lo, hi - (b + 2) / per) : lo;
    *to = fine ? fminf(hi, hi - (b - 2) / per) : hi;
  }
};
static_assert(kBins == 1024, "ten bits");

// Sum over the threads ahead, and of all.
__device__ __forceinline__ unsigned long long block_scan(Shared& sh, unsigned long long x, unsigned long long* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long upto = warp_scan(x);
  if (lane == 31) sh.warp_sum[warp] = upto;
  __syncthreads();
  unsigned long long before = upto - x, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const unsigned long long y = sh.warp_sum[w];
    before += w < warp ? y : 0ULL;
    sum += y;
  }
  __syncthreads();
  *all = sum;
  return before;
}

// A 64-bit sum in shared memory by 32-bit atomics (64-bit ones are a loop of
// compare-and-swap there): whoever sees the low half wrap carries.
__device__ __forceinline__ void add64(unsigned long long* at, unsigned long long x) {
  unsigned int* half = reinterpret_cast<unsigned int*>(at);
  const unsigned int lo = static_cast<unsigned int>(x);
  const unsigned int old = atomicAdd(half, lo);
  const unsigned int hi = static_cast<unsigned int>(x >> 32) + (old + lo < old ? 1u : 0u);
  if (hi != 0) atomicAdd(half + 1, hi);
}

template <typename T>
__device__ __forceinline__ float largest() {  // that T holds
  return sizeof(T) == 2 ? __uint_as_float(0x7F7F0000u) : FLT_MAX;
}

// The CTA's stretch of a row, in shared memory as it came, and -inf up to whole
// cells.  (NaN is in no range and over no threshold.)
template <typename T>
struct Row {
  T* z;
  int cells, first;
  __device__ __forceinline__ void get(int cell, float (&v)[8]) const {
    const int i = cell * kCell + (threadIdx.x & 31) * 8;
    if constexpr (sizeof(T) == 2) {
      const uint4 x = *reinterpret_cast<const uint4*>(z + i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
    } else {
      const float4 x = *reinterpret_cast<const float4*>(z + i), y = *reinterpret_cast<const float4*>(z + i + 4);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    }
  }
  __device__ __forceinline__ int token(int cell, int e) const {
    return first + cell * kCell + static_cast<int>(threadIdx.x & 31) * 8 + e;
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 2) return __bfloat162float(z[i]);
    else return z[i];
  }
  // +inf as the largest number.  (Only where there is one.)
  __device__ __forceinline__ void bound() const {
    for (int i = threadIdx.x; i < cells * kCell; i += kThreads) {
      if constexpr (sizeof(T) == 2) {
        if (__bfloat162float(z[i]) == INFINITY) z[i] = __float2bfloat16(largest<T>());
      } else {
        if (z[i] == INFINITY) z[i] = largest<T>();
      }
    }
    __syncthreads();
  }
};

// n logits into shared memory; this thread's largest.
template <typename T, int VEC>
__device__ __forceinline__ float load_row(const Row<T>& row, const T* from, int n) {
  float top = -INFINITY;
  if constexpr (VEC == 1) {
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const T x = from[i];
      row.z[i] = x;
      top = fmaxf(top, static_cast<float>(x));
    }
  } else {
    static_assert(VEC * sizeof(T) == 16, "16 bytes");
    __nv_bfloat162 pair = __halves2bfloat162(__float2bfloat16(-INFINITY), __float2bfloat16(-INFINITY));
#pragma unroll 4
    for (int i = threadIdx.x * VEC; i < n; i += kThreads * VEC) {  // n is a multiple of VEC
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(from + i));
      *reinterpret_cast<uint4*>(row.z + i) = v;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) pair = __hmax2(pair, *reinterpret_cast<const __nv_bfloat162*>(&w[e]));
        else top = fmaxf(top, __uint_as_float(w[e]));
      }
    }
    if constexpr (sizeof(T) == 2) top = fmaxf(__low2float(pair), __high2float(pair));
  }
  for (int i = n + threadIdx.x; i < row.cells * kCell; i += kThreads) {
    if constexpr (sizeof(T) == 2) row.z[i] = __float2bfloat16(-INFINITY);
    else row.z[i] = -INFINITY;
  }
  return top;
}

// A border's candidates, brought together from the CTAs' parts.
template <int CTAS>
__device__ __forceinline__ void collect(Shared& sh, int n) {
  int i = threadIdx.x;
  if (i < n) {
    int r = 0;
    for (; r < CTAS - 1 && i >= sh.found[r].n; ++r) i -= sh.found[r].n;
    sh.cand[threadIdx.x] = sh.seg[r * (kList / CTAS) + i];
  }
  __syncthreads();
}

__device__ __forceinline__ void clear_bins(Shared& sh) {
  for (int i = threadIdx.x; i < kBins / 2; i += kThreads)
    *reinterpret_cast<uint4*>(&sh.bins[2 * i]) = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

// What a search finds: the value at which the sum by falling value reaches the
// target, the sum over larger values, and the target.  Or `list`: sh.cand has
// all tokens that can be kept (in CTA 0).
struct Border {
  float value;
  unsigned long long above, target;
  int list;
};

// A stretch of logits that a border lies in by all appearances, with its weights in
// sh.bins and the row's in sh.mass, each CTA's own.
struct Window {
  bool is;
  Range range;
};

// The border of the sum of 1 (WEIGHTED false) or of the weights over the row's
// tokens with lo <= z <= hi, by falling z.  target_of(whole sum) gives the
// target, at least 1; where it is past the whole sum the border's value is
// -inf.  All threads of the cluster find the same.  Counts whose tokens down to
// the border are few end as a list.  A border that is not in the window: `list`
// is -1.
template <bool WEIGHTED, int CTAS, typename T, typename F>
__device__ __forceinline__ Border search(cg::cluster_group& cluster, Shared& sh, const Row<T>& row, float lo, float hi,
                                         const Scale& c, F target_of, const Window& window = Window{false, {}}) {
  constexpr int kPart = kList / CTAS;  // candidates from one CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = static_cast<int>(cluster.block_rank());
  unsigned long long above = 0, target = 0;
  Range range;
  for (int level = 0;; ++level) {
    const bool ready = WEIGHTED && level == 0 && window.is;
    if (ready) range = window.range;
    else range.set(lo, hi, level >= 2);
    if (threadIdx.x == 0) sh.n = 0, sh.lo = 0xffffffffu, sh.hi = 0;
    if (!ready) {
      clear_bins(sh);
      for (int cell = warp; cell < row.cells; cell += kWarps) {
        float z[8];
        row.get(cell, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (!range.has(z[e])) continue;
          if constexpr (WEIGHTED) {
            const unsigned long long w = weight(z[e], c, sh.table);
            if (w != 0) add64(&sh.bins[range.bin(z[e])], w);
          } else {
            atomicAdd(reinterpret_cast<unsigned int*>(&sh.bins[range.bin(z[e])]), 1u);
          }
        }
      }
    }
    __syncthreads();
    {  // the groups' sums, to all CTAs: of a group's 16 threads some tell one each
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&sh.bins[2 * threadIdx.x]);
      unsigned long long sum = x.x + x.y;
#pragma unroll
      for (int o = 1; o < kGroup / 2; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int to = lane & (kGroup / 2 - 1);
      if (to < CTAS) cluster.map_shared_rank(&sh, to)->groups[rank][threadIdx.x / (kGroup / 2)] = sum;
    }
    cluster.sync();
    // Every warp finds the border's group; the first one then its bin.
    unsigned long long g = 0, all = 0;
#pragma unroll
    for (int r = 0; r < CTAS; ++r) g += sh.groups[r][lane];
    if (ready) {
#pragma unroll
      for (int r = 0; r < CTAS; ++r) above += sh.mass[r].above, all += sh.mass[r].all;
    }
    const unsigned long long upto = above + warp_scan(g), end = __shfl_sync(0xffffffffu, upto, 31);
    if (level == 0) {
      if (!ready) all = end;
      target = target_of(all);
      if (target > all || target <= above || target > end) {
        cluster.sync();  // all have read the groups
        return Border{-INFINITY, all, target, target > all ? 0 : -1};
      }
    }
    if (warp == 0) {
      const int group = __ffs(__ballot_sync(0xffffffffu, upto >= target)) - 1;
      const unsigned long long before = __shfl_sync(0xffffffffu, upto - g, group);
      unsigned long long b = 0, part[CTAS];
#pragma unroll
      for (int r = 0; r < CTAS; ++r) part[r] = cluster.map_shared_rank(sh.bins, r)[group * kGroup + lane];
#pragma unroll
      for (int r = 0; r < CTAS; ++r) b += part[r];
      const unsigned long long s = before + warp_scan(b);
      const int at = __ffs(__ballot_sync(0xffffffffu, s >= target)) - 1;
      if (lane == at) sh.bin = group * kGroup + lane, sh.above = s - b, sh.in_bin = b;
    }
    __syncthreads();
    const int bin = sh.bin;
    // All tokens down to the border where they are few (counts), else the bin's;
    // and the bin's ends.
    const bool list = !WEIGHTED && level == 0 && sh.above + sh.in_bin <= kList;
    float from, to;
    range.near(bin, &from, &to);
    if (list) to = hi;
    uint32_t l = 0xffffffffu, h = 0;
    for (int cell = warp; cell < row.cells; cell += kWarps) {
      float z[8];
      row.get(cell, z);
      uint32_t in = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) in |= static_cast<uint32_t>(z[e] >= from && z[e] <= to) << e;
      while (in != 0) {  // seldom
        const int e = __ffs(in) - 1;
        in &= in - 1;
        const int i = cell * kCell + lane * 8 + e;
        const float clean = row.at(i) + 0.f;  // -0 is 0
        const int mine = range.bin(clean);
        if (mine > bin || (mine < bin && !list)) continue;
        l = min(l, ordered(clean));
        h = max(h, ordered(clean));
        const int at = atomicAdd(&sh.n, 1), place = rank * kPart + at;
        const Candidate one{clean, row.first + i};
        if (list) {
          (rank == 0 ? sh.cand : sh.seg)[min(at, kList - 1)] = one;  // (they are not more)
          if (rank != 0 && at < kPart) cluster.map_shared_rank(&sh, 0)->seg[place] = one;
        } else if (at < kPart) {
#pragma unroll 1
          for (int r = 0; r < CTAS; ++r) cluster.map_shared_rank(&sh, r)->seg[place] = one;
        }
      }
    }
    l = __reduce_min_sync(0xffffffffu, l);
    h = __reduce_max_sync(0xffffffffu, h);
    if (lane == 0 && h != 0) {
      atomicMin(&sh.lo, l);
      atomicMax(&sh.hi, h);
    }
    __syncthreads();
    if (threadIdx.x < CTAS) cluster.map_shared_rank(&sh, threadIdx.x)->found[rank] = Found{sh.n, sh.lo, sh.hi};
    cluster.sync();
    int n = 0;
    bool fits = true;  // the others' parts
    l = 0xffffffffu, h = 0;
#pragma unroll
    for (int r = 0; r < CTAS; ++r) {
      const Found f = sh.found[r];
      l = min(l, f.lo);
      h = max(h, f.hi);
      n += f.n;
      fits = fits && (f.n <= kPart || (list && r == 0));
    }
    if (list) {
      if (rank == 0) {
        int i = threadIdx.x, r = 0;
        if (i < n) {
          for (; r < CTAS - 1 && i >= sh.found[r].n; ++r) i -= sh.found[r].n;
          if (r > 0) sh.cand[threadIdx.x] = fits ? sh.seg[r * kPart + i] : cluster.map_shared_rank(&sh, r)->seg[i];
        }
        __syncthreads();
      }
      if (!fits) cluster.sync();  // the first CTA has read the others'
      return Border{0.f, 0, target, n};
    }
    above = sh.above;
    lo = unordered(l), hi = unordered(h);
    if (l == h) return Border{hi, above, target, 0};
    if (!fits || n > kFew) continue;
    collect<CTAS>(sh, n);
    if (static_cast<int>(threadIdx.x) < n)
      sh.cand_w[threadIdx.x] = WEIGHTED ? weight(sh.cand[threadIdx.x].z, c, sh.table) : 1ULL;
    __syncthreads();
    // Two threads for each of them: what lies above it, what equals it.
    static_assert(2 * kFew <= kThreads, "two threads a candidate");
    const float mine = sh.cand[min(static_cast<int>(threadIdx.x >> 1), n - 1)].z;
    unsigned long long over = 0, same = 0;
    for (int i = threadIdx.x & 1; i < n; i += 2) {
      const unsigned long long w = sh.cand_w[i];
      over += sh.cand[i].z > mine ? w : 0ULL;
      same += sh.cand[i].z == mine ? w : 0ULL;
    }
    over += above + __shfl_xor_sync(0xffffffffu, over, 1);
    same += __shfl_xor_sync(0xffffffffu, same, 1);
    if (over < target && target <= over + same) sh.value = mine, sh.value_above = over;  // by all its equals alike
    __syncthreads();
    return Border{sh.value, sh.value_above, target, 0};
  }
}

// Looks for the logit at which the weights over `lo` make up `part` of all, by
// counts in bins and the weight in each bin's middle; for the first kSharp bins, whose
// tokens are few and heavy, also by how far off the middle they are.  Then every
// token's weight, once: the sum of all, for every cell the sum (kept: of weights from
// `least` on) of its tokens above a window around that logit, and the window's in
// bins.  The window is 2 bins either way: of 5000 rows drawn (normal logits, some
// likely ones among them, in bf16 and fp32) the border was 1.8 off at most; without
// the first bins' offsets, 0.4% were off by more than 3.5.  Of 34000 rows of other
// shapes (power laws, exponential, groups, masked; temperatures of 0.1 to 4; top-p
// 0.3 to 0.999) 26 missed it, of one shape at one temperature (rank^-3, 1.5) 3 of
// 150: where the border lies at a gap.  It is searched for again then without a
// window: 128 rows of 50021, all of which miss it, take 73 us against 50.
constexpr int kSharp = 256;
template <int CTAS, typename T>
__device__ __forceinline__ Window look(cg::cluster_group& cluster, Shared& sh, const Row<T>& row, float lo, float top,
                                       const Scale& c, float part, unsigned long long least) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = static_cast<int>(cluster.block_rank());
  Range range;
  range.set(lo, top, false);
  clear_bins(sh);
  unsigned int* counts = reinterpret_cast<unsigned int*>(sh.bins);
  static_assert(kBins + kSharp <= 2 * kBins, "room beside the counts");
  int* offsets = reinterpret_cast<int*>(sh.bins) + kBins;
  for (int cell = warp; cell < row.cells; cell += kWarps) {
    float z[8];
    row.get(cell, z);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!range.has(z[e])) continue;
      const int b = range.bin(z[e]);
      atomicAdd(&counts[b], 1u);
      if (b < kSharp) atomicAdd(&offsets[b], range.offset(z[e], b));
    }
  }
  __syncthreads();
  const float step = -c.hi / range.per * c.by;  // log2 of the weights from bin to bin
  const float per_offset = step * 0.693147181f / Range::kOffset;
  {
    const int b = 2 * static_cast<int>(threadIdx.x);
    float n0 = counts[b], n1 = counts[b + 1];
    if (b < kSharp) n0 += offsets[b] * per_offset, n1 += offsets[b + 1] * per_offset;
    float sum = n0 * ex2(b * step) + n1 * ex2((b + 1) * step);
#pragma unroll
    for (int o = 1; o < kGroup / 2; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int to = lane & (kGroup / 2 - 1);
    if (to < CTAS)
      reinterpret_cast<float*>(cluster.map_shared_rank(&sh, to)->groups[rank])[threadIdx.x / (kGroup / 2)] = sum;
  }
  cluster.sync();
  if (warp == 0) {
    float g = 0.f;
#pragma unroll
    for (int r = 0; r < CTAS; ++r) g += reinterpret_cast<const float*>(sh.groups[r])[lane];
    const float upto = warp_scan(g);
    const float want = part * __shfl_sync(0xffffffffu, upto, 31);
    const uint32_t over = __ballot_sync(0xffffffffu, upto >= want);
    const int group = over != 0 ? __ffs(over) - 1 : 31;
    const float before = __shfl_sync(0xffffffffu, upto - g, group);
    const int b = group * kGroup + lane;
    const bool sharp = group < kSharp / kGroup;
    unsigned int n[CTAS], whole = 0;
    int off[CTAS], off_middle = 0;
#pragma unroll
    for (int r = 0; r < CTAS; ++r) {
      const unsigned int* other = reinterpret_cast<const unsigned int*>(cluster.map_shared_rank(sh.bins, r));
      n[r] = other[b];
      off[r] = sharp ? static_cast<int>(other[kBins + b]) : 0;
    }
#pragma unroll
    for (int r = 0; r < CTAS; ++r) whole += n[r], off_middle += off[r];
    const float count = whole + off_middle * per_offset;
    const uint32_t past = __ballot_sync(0xffffffffu, before + warp_scan(count * ex2(b * step)) >= want);
    if (lane == 0) sh.bin = group * kGroup + (past != 0 ? __ffs(past) - 1 : 31);
  }
  cluster.sync();  // all have read the others' counts
  const float from = fmaxf(lo, top - (sh.bin + 2) / range.per), to = fminf(top, top - (sh.bin - 2) / range.per);
  Window window{true, {}};
  window.range.set(from, to, false);
  clear_bins(sh);
  unsigned long long all = 0, above = 0;
  for (int cell = warp; cell < row.cells; cell += kWarps) {
    unsigned long long over = 0, less = 0;  // above the window; of those, what min_p does not keep
    float z[8];
    row.get(cell, z);
#pragma unroll
    for (int half = 0; half < 8; half += 4) {
      unsigned long long w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = weight(z[half + e], c, sh.table);
        w[e] = z[half + e] >= lo ? w[e] : 0ULL;
        all += w[e];
        over += z[half + e] > to ? w[e] : 0ULL;
      }
      if (least != 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) less += z[half + e] > to && w[e] < least ? w[e] : 0ULL;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (z[half + e] >= from && z[half + e] <= to) add64(&sh.bins[window.range.bin(z[half + e])], w[e]);
    }
    above += over;
    unsigned long long kept = over - less;
    if (__any_sync(0xffffffffu, kept != 0)) kept = warp_sum(kept);
    if (lane == 0) sh.cell_over[cell] = kept;
  }
  block_scan(sh, all, &all);
  block_scan(sh, above, &above);
  if (threadIdx.x < CTAS) cluster.map_shared_rank(&sh, threadIdx.x)->mass[rank] = Mass{all, above};
  return window;
}

struct Settings {
  int top_k;
  float top_p;               // 1: off
  unsigned long long least;  // the smallest weight that min_p keeps
  float u;
};

__device__ __forceinline__ unsigned long long drawn(float u, unsigned long long whole) {
  return u >= 1.f ? whole - 1 : u > 0.f ? share_of(u, whole, false) : 0ULL;
}
__device__ __forceinline__ void put(const SampleArgs& p, int b, int token, unsigned long long w,
                                    unsigned long long whole) {
  p.tokens[b] = token;
  if (p.prob != nullptr) p.prob[b] = whole != 0 ? __ull2float_rn(w) / __ull2float_rn(whole) : 0.f;
}

// The keys of the first n threads sorted: thread t's is the t-th.  Only the largest
// number, which is behind all and which the others have, may come twice.  Few are
// counted each with each, four or two threads a key; more go through Batcher's
// bitonic network, whose 45 steps for 512 keys each wait for the one before: by top-k
// 50 and 120 of a row of 32768 the whole call takes 8.4 and 9.0 us counted, 9.8 and
// 10.7 by the network, which for 400 takes 12.9, counted 17.2.
__device__ __forceinline__ unsigned long long sort_keys(Shared& sh, unsigned long long key, int n) {
  static_assert(kList <= kThreads && 2 * kList <= kBins, "a thread a key, two buffers in the bins, which have served");
  const int t = static_cast<int>(threadIdx.x);
  if (n <= kCounted) {
    static_assert(2 * kCounted <= kThreads, "two threads a key, or four");
    const int log = n <= kThreads / 4 ? 2 : 1, mine = t >> log, part = t & ((1 << log) - 1);
    if (t < n) sh.bins[t] = key, sh.bins[kList + t] = ~0ULL;
    __syncthreads();
    const unsigned long long me = sh.bins[min(mine, n - 1)];
    int less = 0;
#pragma unroll 4
    for (int i = part; i < n; i += 1 << log) less += sh.bins[i] < me;
    less += __shfl_xor_sync(0xffffffffu, less, 1);
    if (log == 2) less += __shfl_xor_sync(0xffffffffu, less, 2);
    if (part == 0 && mine < n) sh.bins[kList + less] = me;
    __syncthreads();
    return t < n ? sh.bins[kList + t] : ~0ULL;
  }
  int size = 2 * kCounted, buffer = 0;
  while (size < n) size <<= 1;
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      unsigned long long other;
      if (j >= 32) {
        sh.bins[buffer + t] = key;
        __syncthreads();
        other = sh.bins[buffer + (t ^ j)];
        buffer ^= kList;
      } else {
        other = __shfl_xor_sync(0xffffffffu, key, j);
      }
      const bool least = ((t & k) == 0) == ((t & j) == 0);
      key = (other < key) == least ? other : key;
    }
  return key;
}

// The token of one of n <= kList candidates, by one CTA: sorted by falling logit,
// equal ones by index, for the filters; then by index, for the draw.
__device__ __forceinline__ void finish_list(Shared& sh, int n, const Settings& set, const Scale& c,
                                            const SampleArgs& p, int b) {
  static_assert(kSampleMaxVocab <= 1 << 18 && kOne == 44, "a token and its weight fit 63 bits");
  const int t = static_cast<int>(threadIdx.x);
  unsigned long long key = ~0ULL;
  if (t < n) {
    const Candidate me = sh.cand[t];
    key = static_cast<unsigned long long>(~ordered(me.z)) << 32 | static_cast<uint32_t>(me.token);
  }
  __syncthreads();
  key = sort_keys(sh, key, n);
  const unsigned long long x =
      t < n && t < set.top_k ? weight(unordered(~static_cast<uint32_t>(key >> 32)), c, sh.table) : 0ULL;
  unsigned long long all;
  const unsigned long long before = block_scan(sh, x, &all);
  const unsigned long long target =
      set.top_p < 1.f ? (set.top_p > 0.f ? max(1ULL, share_of(set.top_p, all, true)) : 1ULL) : all;
  const bool kept = before < target && x >= set.least && x != 0;
  key = sort_keys(sh, kept ? (key & 0xffffffffu) << (kOne + 1) | x : ~0ULL, n);
  const unsigned long long y = key != ~0ULL ? key & ((2ULL << kOne) - 1) : 0ULL;
  unsigned long long whole;
  const unsigned long long from = block_scan(sh, y, &whole);
  const unsigned long long at = drawn(set.u, whole);
  if (from <= at && at < from + y) put(p, b, static_cast<int>(key >> (kOne + 1)), y, whole);
}

template <typename T, int VEC, int CTAS>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs p, int stretch) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = static_cast<int>(blockIdx.y);
  const int n_row = max(0, min(stretch, p.V - rank * stretch));
  const Row<T> row{reinterpret_cast<T*>(smem + sizeof(Shared)), (n_row + kCell - 1) / kCell, rank * stretch};
  cluster.barrier_arrive();  // a CTA that runs may be written to
  grid_dep_wait();
  grid_dep_launch_dependents();
  const float temperature = p.temperature != nullptr ? __ldg(p.temperature + b) : 1.f;
  const int k_asked = p.top_k != nullptr ? __ldg(p.top_k + b) : 0;
  const float p_asked = p.top_p != nullptr ? __ldg(p.top_p + b) : 1.f;
  const float m_asked = p.min_p != nullptr ? __ldg(p.min_p + b) : 0.f;
  Settings set;
  set.u = __ldg(p.uniform + b);
  for (int i = threadIdx.x; i < kTable; i += kThreads) sh.table[i] = kPowers.v[i];
  float top = load_row<T, VEC>(row, static_cast<const T*>(p.logits) + b * p.row_stride + row.first, n_row);
  const bool greedy = !(temperature > 0.f);
  set.top_k = greedy ? 1 : k_asked;
  set.top_p = !greedy && p_asked < 1.f ? p_asked : 1.f;
  set.least = !greedy && m_asked > 0.f ? __float2ull_ru(fminf(m_asked, 1.f) * 0x1p44f) : 0ULL;

  // The row's largest logit.  And one that is not over the top_k-th largest,
  // without which the search would put the whole row into bins: of `parts` parts
  // of the row, at least top_k, the smallest of their largest.  (A part is a
  // thread's logits or several threads'; parts without any do not count.)  Where
  // there are too few threads, the smallest logit.
  float cut = top;
  int parts = 0;
  {
    const int busy = CTAS * min(kThreads, (min(stretch, p.V) + VEC - 1) / VEC);  // of the row, about
    int o = 32;  // threads of a part
    while (o > 1 && busy / o < set.top_k) o >>= 1;
    for (int x = 1; x < o; x <<= 1) cut = fmaxf(cut, __shfl_xor_sync(0xffffffffu, cut, x));
    if (busy < set.top_k) {
      __syncthreads();
      cut = INFINITY;
      for (int i = threadIdx.x; i < row.cells * kCell; i += kThreads) {
        const float z = row.at(i);
        if (z > -INFINITY) cut = fminf(cut, z);
      }
      parts = 1 << 20;
    } else {
      parts = __popc(__ballot_sync(0xffffffffu, cut > -INFINITY && (lane & (o - 1)) == 0));
      if (cut == -INFINITY) cut = INFINITY;
    }
    const uint32_t l = __reduce_min_sync(0xffffffffu, ordered(cut)), h = __reduce_max_sync(0xffffffffu, ordered(top));
    if (lane == 0) sh.warp_cut[warp] = l, sh.warp_top[warp] = unordered(h), sh.warp_parts[warp] = parts;
  }
  __syncthreads();
  cluster.barrier_wait();
  if (warp == 0) {
    const uint32_t l = __reduce_min_sync(0xffffffffu, lane < kWarps ? sh.warp_cut[lane] : 0xffffffffu);
    const uint32_t h = __reduce_max_sync(0xffffffffu, lane < kWarps ? ordered(sh.warp_top[lane]) : 0u);
    const int n = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_parts[lane] : 0);
    if (lane < CTAS) {
      Shared* other = cluster.map_shared_rank(&sh, lane);
      other->top[rank] = unordered(h);
      other->cut[rank] = l;
      other->parts[rank] = n;
    }
  }
  cluster.sync();
  uint32_t cut_at = 0xffffffffu;
  parts = 0;
#pragma unroll
  for (int r = 0; r < CTAS; ++r) {
    top = r == 0 ? sh.top[0] : fmaxf(top, sh.top[r]);
    cut_at = min(cut_at, sh.cut[r]);
    parts += sh.parts[r];
  }
  if (top == -INFINITY) {
    if (rank == 0 && threadIdx.x == 0) put(p, b, -1, 0, 0);
    return;  // the whole cluster
  }
  top += 0.f;  // -0 is 0
  if (top == INFINITY) {
    row.bound();
    top = largest<T>();
  }
  cut = parts >= set.top_k ? fminf(unordered(cut_at), top) : -INFINITY;
  const Scale c = greedy ? Scale{0.f, 0.f, top, 1.f} : scale_of(temperature, top);

  // The threshold: tokens over `value`, and the first `ties` of those at it.
  float value = -INFINITY;
  long long ties = 0;
  float counted = INFINITY;  // cell_over has the tokens over it
  if (set.top_k == 1) {
    value = top, ties = 1;
  } else if (set.top_k > 0 && set.top_k < p.V) {
    const auto target_of = [&](unsigned long long) { return static_cast<unsigned long long>(set.top_k); };
    const Border k = search<false, CTAS>(cluster, sh, row, fmaxf(cut, -FLT_MAX), top, c, target_of);
    if (k.list > 0) {
      if (rank == 0) finish_list(sh, k.list, set, c, p, b);
      return;
    }
    value = k.value;  // -inf: there are no more than top_k
    ties = value == -INFINITY ? 0 : static_cast<long long>(k.target - k.above);
  }
  if (set.top_p < 1.f) {
    // The smallest part of what is left that makes up top_p of it.
    const unsigned long long at_value = ties > 0 ? ties * weight(value, c, sh.table) : 0ULL;
    const auto target_of = [&](unsigned long long all) {
      return set.top_p > 0.f ? max(1ULL, share_of(set.top_p, all + at_value, true)) : 1ULL;
    };
    unsigned long long above = 0, target;
    float at = -INFINITY;
    if (value < top) {
      const float reach = top - 45.5f / c.hi / c.by;  // below, weights are 0
      const float next = value == -INFINITY ? -FLT_MAX : unordered(ordered(value) + 1);
      const float lo = fmaxf(next, reach);
      Border s{0.f, 0, 0, -1};
      if (value == -INFINITY) {
        const Window window = look<CTAS>(cluster, sh, row, lo, top, c, set.top_p, set.least);
        s = search<true, CTAS>(cluster, sh, row, lo, top, c, target_of, window);
        if (s.list == 0) counted = window.range.hi;
      }
      if (s.list < 0) s = search<true, CTAS>(cluster, sh, row, lo, top, c, target_of);
      at = s.value, above = s.above, target = s.target;
    } else {
      target = target_of(0);
    }
    // (Rounded up; none of the weights that the sums count is 0.)
    const unsigned long long w = weight(at == -INFINITY ? value : at, c, sh.table);
    const long long need = static_cast<long long>((target - above + w - 1) / w);
    ties = at == -INFINITY ? min(ties, need) : need;
    value = at == -INFINITY ? value : at;
  }
  const unsigned long long w_tie = ties > 0 ? weight(value, c, sh.table) : 0ULL;
  if (w_tie < set.least) ties = 0;

  // The kept weights of every cell, then of the CTA, then of the row.
  const auto kept_weight = [&](float z) {
    const unsigned long long w = z > value ? weight(z, c, sh.table) : 0ULL;
    return w < set.least ? 0ULL : w;
  };
  for (int cell = warp; cell < row.cells; cell += kWarps) {
    unsigned long long w = 0;
    int at = 0;
    float z[8];
    row.get(cell, z);
    if (value == -INFINITY) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w += kept_weight(z[e]);
    } else {
      uint32_t in = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        in |= static_cast<uint32_t>(z[e] > value && z[e] <= counted) << e;
        at += z[e] == value;
      }
      for (; in != 0; in &= in - 1) w += kept_weight(row.at(cell * kCell + lane * 8 + __ffs(in) - 1));  // few
    }
    if (__any_sync(0xffffffffu, w != 0)) w = warp_sum(w);
    at = __reduce_add_sync(0xffffffffu, at);
    if (lane == 0) {
      if (counted < INFINITY) w += sh.cell_over[cell];
      sh.cell_over[cell] = w;
      sh.cell_ties[cell] = at;
    }
  }
  __syncthreads();
  // The first warp goes on with kLaneCells cells a lane, and what lies ahead of them.
  unsigned long long over[kLaneCells], over_before = 0;
  int at[kLaneCells], at_before = 0;
  if (warp == 0) {
    unsigned long long sum = 0;
    int sum_at = 0;
#pragma unroll
    for (int i = 0; i < kLaneCells; ++i) {
      const bool is = kLaneCells * lane + i < row.cells;
      over[i] = is ? sh.cell_over[kLaneCells * lane + i] : 0ULL;
      at[i] = is ? sh.cell_ties[kLaneCells * lane + i] : 0;
      sum += over[i];
      sum_at += at[i];
    }
    const unsigned long long upto = warp_scan(sum);
    const int at_upto = warp_scan(sum_at);
    over_before = upto - sum;
    at_before = at_upto - sum_at;
    const Kept all{__shfl_sync(0xffffffffu, upto, 31), __shfl_sync(0xffffffffu, at_upto, 31)};
    if (lane < CTAS) cluster.map_shared_rank(&sh, lane)->kept[rank] = all;
  }
  cluster.sync();  // the last: nobody writes to another CTA from here on
  if (warp != 0) return;
  const auto kept = [](long long left, int n) {
    return static_cast<unsigned long long>(min(left, static_cast<long long>(n)));
  };
  unsigned long long whole = 0, ahead = 0;
  long long ties_left = 0, left = ties;  // for this CTA and those behind it
#pragma unroll
  for (int r = 0; r < CTAS; ++r) {
    const Kept other = sh.kept[r];
    if (r == rank) ahead = whole, ties_left = left;
    const unsigned long long take = kept(left, other.ties);
    whole += other.over + take * w_tie;
    left -= static_cast<long long>(take);
  }
  const unsigned long long target = drawn(set.u, whole);  // the token's running sum is the first over it
  // The cell, in this CTA or another; then the token.
  int cell = -1, cell_at = 0;
  unsigned long long rest = 0;
#pragma unroll
  for (int i = 0; i < kLaneCells; ++i) {
    const unsigned long long from = ahead + over_before + kept(ties_left, at_before) * w_tie;
    const int before = at_before;
    over_before += over[i];
    at_before += at[i];
    const unsigned long long to = ahead + over_before + kept(ties_left, at_before) * w_tie;
    if (from <= target && target < to) cell = kLaneCells * lane + i, cell_at = before, rest = target - from;
  }
  const uint32_t who = __ballot_sync(0xffffffffu, cell >= 0);
  if (who == 0) return;
  cell = __shfl_sync(0xffffffffu, cell, __ffs(who) - 1);
  cell_at = __shfl_sync(0xffffffffu, cell_at, __ffs(who) - 1);
  rest = __shfl_sync(0xffffffffu, rest, __ffs(who) - 1);
  float z[8];
  row.get(cell, z);
  unsigned long long w[8], sum = 0;
  int n_at = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) n_at += z[e] == value;
  int rank_at = cell_at + warp_scan(n_at) - n_at;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = kept_weight(z[e]);
    if (z[e] == value) w[e] = rank_at++ < ties_left ? w_tie : 0ULL;
    sum += w[e];
  }
  unsigned long long from = warp_scan(sum) - sum;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (from <= rest && rest < from + w[e]) put(p, b, row.token(cell, e), w[e], whole);
    from += w[e];
  }
}

// Of type T, with all else that a CTA has in shared memory.
template <typename T>
constexpr int max_cells() {
  return std::min(kCells, static_cast<int>((227 * 1024 - sizeof(Shared)) / (kCell * sizeof(T))));
}
static_assert(kSampleMaxVocab <= kMaxCluster * max_cells<float>() * kCell, "a cluster has room for a row");

template <typename T, int VEC, int CTAS>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream) {
  const int stretch = ((a.V + CTAS - 1) / CTAS + kCell - 1) / kCell * kCell;
  const size_t smem = sizeof(Shared) + static_cast<size_t>(stretch) * sizeof(T);
  auto kernel = sample_kernel<T, VEC, CTAS>;
  // The most that any call needs: another thread may set it at the same time.
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       sizeof(Shared) + max_cells<T>() * kCell * sizeof(T));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CTAS, a.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, stretch);
}

template <typename T, int VEC>
cudaError_t by_size(const SampleArgs& a, cudaStream_t stream) {
  // CTAs of a row, by the time that they take: fitted to 220 measured ones (1 to 256
  // rows of 4096 to 131072, bf16 and fp32, with and without top-k and top-p), whose
  // best it misses by 1% on average and 18% at most.  Some rows find room at a time,
  // two CTAs on an SM where their stretches fit, the others follow.  Both ends, by
  // top-p: one row of 131072 takes 25 us by 8 CTAs and 60 by 2, 256 of 16384 take 36
  // by one each and 121 by 8.  (Fitted with room for one cluster of 4 and three of 8
  // more than there is; where that decides, the true counts give, by top-p and by
  // top-k: 37 rows of 131072 in fp32 56 us for 70 and 22 for 20.5, 148 of them 167
  // for 185 and 58 both, 16 of 185364 51 for 60 and 15 for 20.)
  int ctas = 0;
  double best = 0;
  for (int log = 0; 1 << log <= kMaxCluster; ++log) {
    const int c = 1 << log, stretch = ((a.V + c - 1) / c + kCell - 1) / kCell * kCell;
    if (stretch > max_cells<T>() * kCell) continue;
    const bool two = 2 * (sizeof(Shared) + stretch * sizeof(T) + 1024) <= 228 * 1024;
    const int places = clusters_at_a_time(log, two ? 2 : 1), rest = a.B % places;
    const auto us = [&](bool shared) { return 10 + 1.5 * log + stretch / 1200.0 * (shared ? 1.9 : 1.0); };
    const double all = a.B / places * us(two) + (rest == 0 ? 0.0 : us(two && rest > places / 2));
    if (ctas == 0 || all < best) ctas = c, best = all;
  }
  switch (ctas) {
    case 1: return launch<T, VEC, 1>(a, stream);
    case 2: return launch<T, VEC, 2>(a, stream);
    case 4: return launch<T, VEC, 4>(a, stream);
    case 8: return launch<T, VEC, 8>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream) {
  const int vec = a.bf16 ? 8 : 4;
  const bool on16 = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.V % vec == 0 &&
                    (a.row_stride % vec == 0 || a.B == 1);
  if (a.bf16) return on16 ? by_size<__nv_bfloat16, 8>(a, stream) : by_size<__nv_bfloat16, 1>(a, stream);
  return on16 ? by_size<float, 4>(a, stream) : by_size<float, 1>(a, stream);
}

}  // namespace txl
