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
// the largest weight (to about 2^-39 of its own size) and 64-bit sums of at most
// 2^18 of them do not depend on their order.  In fp32, sums over 100000 tokens
// would name another token once in a hundred rows or so; in fp64 the
// exponentials alone would take many times the kernel's time on this chip.
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
constexpr int kBins = 2048;
constexpr int kFew = 512;        // tokens of a bin that are compared each with each
constexpr int kMaxCluster = 8;
constexpr int kTable = 512;      // steps of the powers' table
constexpr int kOne = 44;         // the largest weight is 2^kOne
constexpr unsigned long long kUnit = 1ULL << kOne;
constexpr int kCells = 1024;

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

struct Scale {  // log2(e) / T in two parts
  float hi, lo;
};

// exp((z - top) / T) in units of 2^-44.  With y = (top - z) log2(e) / T as the
// sum of two floats, y = k / 512 + r, the weight is 2^-(k/512), from the table,
// times 1 - q, q = 1 - 2^-r by its series in whole numbers of 2^-40: |r| <=
// 2^-10, so three terms do.
__device__ __forceinline__ unsigned long long weight(float z, float top, Scale c, const unsigned long long* table) {
  float d = top - z;
  const float back = d - top;
  float err = (top - (d - back)) - (z + back);  // top - z = d + err
  if (d > 3.0e38f) d = FLT_MAX, err = 0.f;
  const float y = d * c.hi;
  const float y2 = fmaf(d, c.hi, -y) + fmaf(d, c.lo, err * c.hi);
  if (!(y < 45.f)) return 0;
  const float kf = rintf(y * kTable);
  const float f = fmaf(kf, -1.f / kTable, y);
  const int k = static_cast<int>(kf);
  const int r = __float2int_rn(f * 0x1p40f) + __float2int_rn(y2 * 0x1p40f);
  // ln 2 in units of 2^-31
  const int x = static_cast<int>((static_cast<long long>(r) * 1488522236LL + (1LL << 30)) >> 31);
  const int x2 = static_cast<int>((static_cast<long long>(x) * x) >> 41);      // x^2 / 2
  const int x3 = static_cast<int>((static_cast<long long>(x2) * x) >> 40) / 3;  // x^3 / 6
  const int q = x - x2 + x3;
  const unsigned long long p = table[k & (kTable - 1)];
  const int p31 = static_cast<int>(min(p >> (kOne - 31), 0x7fffffffULL));
  const long long less = (static_cast<long long>(q) * p31) >> (31 - (kOne - 40));
  return static_cast<unsigned long long>(static_cast<long long>(p) - less) >> (k / kTable);
}

// A float's place in the order of floats, as a whole number.
__device__ __forceinline__ uint32_t ordered(float z) {
  const uint32_t u = __float_as_uint(z);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

struct Shared {
  unsigned long long table[kTable];
  unsigned long long bins[kBins];  // of the range at hand: sums of weights, or counts
  // A bin's tokens: how many of this CTA, their ends (ordered), the first of
  // them; then the cluster's, with their weights (or 1).
  int found;
  uint32_t lo, hi;
  float mine[kFew];
  float cand[kFew];
  unsigned long long cand_w[kFew];
  unsigned long long warp_sum[kWarps];
  int warp_ties[kWarps];
  int live;
  Scale scale;
  int bin;                   // where the border lies,
  unsigned long long above;  // and the sum ahead of it
  float value;
  unsigned long long value_above;
  // The last step: weights over the threshold and tokens at it, of this CTA and
  // of its cells (the tokens that a warp loads at once).
  unsigned long long over;
  int ties;
  int cell;
  unsigned long long rest;
  int ties_before;
  unsigned long long cell_over[kCells];
  int cell_ties[kCells];
};

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

// The bins of a range of logits, largest first.  Linear between its ends, in
// halves so that no difference overflows; by the floats' order where `keys`
// (for ranges that the linear map does not separate).
struct Range {
  float lo, hi;
  bool keys;
  int shift;
  float inv;
  __device__ __forceinline__ void set(float l, float h, bool k) {
    lo = l, hi = h, keys = k;
    const uint32_t span = ordered(h) - ordered(l);
    shift = max(0, 32 - __clz(span) - 11);
    inv = kBins / (0.5f * h - 0.5f * l);
  }
  __device__ __forceinline__ bool has(float z) const { return z >= lo && z <= hi; }
  __device__ __forceinline__ int bin(float z) const {
    if (keys) return static_cast<int>((ordered(hi) - ordered(z)) >> shift);
    return static_cast<int>(fminf((0.5f * hi - 0.5f * z) * inv, kBins - 1.f));  // (0 * inf: NaN, bin 0 or the last)
  }
};

// What a search finds: the value at which the sum by falling value reaches the
// target, the sum over larger values, and the target.
struct Border {
  float value;
  unsigned long long above, target;
};

// The CTA's stretch of a row, in shared memory: -inf in place of NaN, the
// largest float of +inf, 0 of -0.
struct Row {
  float* z;
  int n;

  template <typename T, int VEC>
  __device__ __forceinline__ void load(const T* from) const {
    const auto clean = [](float x) { return isnan(x) ? -INFINITY : fminf(x + 0.f, FLT_MAX); };
    if constexpr (VEC == 1) {
#pragma unroll 8
      for (int i = threadIdx.x; i < n; i += kThreads) {
        if constexpr (sizeof(T) == 2) z[i] = clean(__bfloat162float(from[i]));
        else z[i] = clean(from[i]);
      }
    } else {
      static_assert(VEC * sizeof(T) == 16, "16 bytes");
#pragma unroll 4
      for (int i = threadIdx.x * VEC; i < n; i += kThreads * VEC) {  // n is a multiple of VEC
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(from + i));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          z[i + e] = clean(sizeof(T) == 4 ? __uint_as_float(w[e % 4]) : e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]));
      }
    }
  }
};

// The border of the sum of 1 (WEIGHTED false) or of the weights over the row's
// tokens with lo <= z <= hi, by falling z.  target_of(whole sum) gives the
// target, at least 1; where it is past the whole sum the border's value is
// -inf.  All threads of the cluster find the same.
template <bool WEIGHTED, typename F>
__device__ __forceinline__ Border search(cg::cluster_group& cluster, Shared& sh, const Row& row, float lo, float hi,
                                         float top, Scale c, F target_of) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctas = static_cast<int>(cluster.num_blocks());
  unsigned long long above = 0, target = 0;
  Range range;
  for (int level = 0;; ++level) {
    range.set(lo, hi, level >= 2);
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.bins[i] = 0;
    if (threadIdx.x == 0) sh.found = 0, sh.lo = 0xffffffffu, sh.hi = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
      const float z = row.z[i];
      if (!range.has(z)) continue;
      if constexpr (WEIGHTED) {
        const unsigned long long w = weight(z, top, c, sh.table);
        if (w != 0) atomicAdd(&sh.bins[range.bin(z)], w);
      } else {
        atomicAdd(reinterpret_cast<unsigned int*>(&sh.bins[range.bin(z)]), 1u);
      }
    }
    cluster.sync();
    // Every CTA adds up the bins of all: a few in a line per thread.
    constexpr int kPer = kBins / kThreads;
    unsigned long long b[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) b[i] = 0;
    for (int r = 0; r < ctas; ++r) {
      const unsigned long long* from = cluster.map_shared_rank(sh.bins, r) + threadIdx.x * kPer;
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(from + i);
        b[i] += v.x;
        b[i + 1] += v.y;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += b[i];
    const unsigned long long upto = warp_scan(sum);
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    unsigned long long before = above, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const unsigned long long x = sh.warp_sum[w];
      before += w < warp ? x : 0ULL;
      all += x;
    }
    before += upto - sum;
    if (level == 0) {
      target = target_of(all);
      if (target > all) {
        cluster.sync();  // all have read the bins
        return Border{-INFINITY, all, target};
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (before < target && target <= before + b[i]) sh.bin = threadIdx.x * kPer + i, sh.above = before;
      before += b[i];
    }
    __syncthreads();
    const int bin = sh.bin;
    above = sh.above;
    // The bin's tokens: their ends, and the tokens where they are few.
    uint32_t l = 0xffffffffu, h = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
      const float z = row.z[i];
      if (!range.has(z) || range.bin(z) != bin) continue;
      l = min(l, ordered(z));
      h = max(h, ordered(z));
      const int at = atomicAdd(&sh.found, 1);
      if (at < kFew) sh.mine[at] = z;
    }
    l = __reduce_min_sync(0xffffffffu, l);
    h = __reduce_max_sync(0xffffffffu, h);
    if (lane == 0 && h != 0) {
      atomicMin(&sh.lo, l);
      atomicMax(&sh.hi, h);
    }
    cluster.sync();
    int n = 0;
    l = 0xffffffffu, h = 0;
    for (int r = 0; r < ctas; ++r) {
      const Shared* other = cluster.map_shared_rank(&sh, r);
      l = min(l, other->lo);
      h = max(h, other->hi);
      n += other->found;
    }
    lo = unordered(l), hi = unordered(h);
    const bool one = l == h, few = n <= kFew;
    if (!one && few) {
      int at = 0;
      for (int r = 0; r < ctas; ++r) {
        const Shared* other = cluster.map_shared_rank(&sh, r);
        const int m = other->found;
        for (int i = threadIdx.x; i < m; i += kThreads) {
          const float z = other->mine[i];
          sh.cand[at + i] = z;
          sh.cand_w[at + i] = WEIGHTED ? weight(z, top, c, sh.table) : 1ULL;
        }
        at += m;
      }
    }
    cluster.sync();  // all have read: bins, found and mine may be written again
    if (one) return Border{hi, above, target};
    if (!few) continue;
    static_assert(kFew <= kThreads, "a candidate a thread");
    if (static_cast<int>(threadIdx.x) < n) {
      const float mine = sh.cand[threadIdx.x];
      unsigned long long a = above, same = 0;
      for (int i = 0; i < n; ++i) {
        const unsigned long long w = sh.cand_w[i];
        a += sh.cand[i] > mine ? w : 0ULL;
        same += sh.cand[i] == mine ? w : 0ULL;
      }
      if (a < target && target <= a + same) sh.value = mine, sh.value_above = a;  // by all its equals alike
    }
    __syncthreads();
    return Border{sh.value, sh.value_above, target};
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs p, int stretch) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = static_cast<int>(blockIdx.y);
  const int first = rank * stretch;
  const Row row{reinterpret_cast<float*>(smem + sizeof(Shared)), max(0, min(stretch, p.V - first))};
  grid_dep_wait();
  grid_dep_launch_dependents();
  row.load<T, VEC>(static_cast<const T*>(p.logits) + b * p.row_stride + first);
  for (int i = threadIdx.x; i < kTable; i += kThreads) sh.table[i] = kPowers.v[i];
  const float temperature = p.temperature != nullptr ? __ldg(p.temperature + b) : 1.f;
  const bool greedy = !(temperature > 0.f);
  const int top_k = greedy ? 1 : p.top_k != nullptr ? __ldg(p.top_k + b) : 0;
  const float top_p = !greedy && p.top_p != nullptr ? __ldg(p.top_p + b) : 1.f;
  const float min_p = !greedy && p.min_p != nullptr ? __ldg(p.min_p + b) : 0.f;
  if (threadIdx.x == 0) {
    const double x = greedy ? 0.0 : 1.4426950408889634 / static_cast<double>(temperature);
    const float hi = fminf(static_cast<float>(x), FLT_MAX);
    sh.scale = Scale{hi, hi < FLT_MAX ? static_cast<float>(x - static_cast<double>(hi)) : 0.f};
    sh.lo = 0xffffffffu, sh.hi = 0, sh.live = 0;
  }
  __syncthreads();
  const Scale c = sh.scale;

  // The row's largest and smallest logit, how many it has.
  {
    uint32_t l = 0xffffffffu, h = 0;
    int live = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
      const float z = row.z[i];
      if (z == -INFINITY) continue;
      l = min(l, ordered(z));
      h = max(h, ordered(z));
      ++live;
    }
    l = __reduce_min_sync(0xffffffffu, l);
    h = __reduce_max_sync(0xffffffffu, h);
    live = __reduce_add_sync(0xffffffffu, live);
    if (lane == 0 && live > 0) {
      atomicMin(&sh.lo, l);
      atomicMax(&sh.hi, h);
      atomicAdd(&sh.live, live);
    }
  }
  cluster.sync();
  uint32_t l = 0xffffffffu, h = 0;
  int live = 0;
  for (int r = 0; r < ctas; ++r) {
    const Shared* other = cluster.map_shared_rank(&sh, r);
    l = min(l, other->lo);
    h = max(h, other->hi);
    live += other->live;
  }
  cluster.sync();
  if (live == 0) {
    if (rank == 0 && threadIdx.x == 0) {
      p.tokens[b] = -1;
      if (p.prob != nullptr) p.prob[b] = 0.f;
    }
    return;  // the whole cluster
  }
  const float top = unordered(h), bottom = unordered(l);

  // The threshold: tokens over `value`, and the first `ties` of those at it.
  float value = -INFINITY;
  long long ties = 0;
  if (top_k == 1) {
    value = top, ties = 1;
  } else if (top_k > 0 && top_k < live) {
    const Border k = search<false>(cluster, sh, row, bottom, top, top, c,
                                   [&](unsigned long long) { return static_cast<unsigned long long>(top_k); });
    value = k.value;
    ties = static_cast<long long>(k.target - k.above);
  }
  if (top_p < 1.f && value < top) {
    // The smallest share of the whole that holds top_p of it.
    const unsigned long long at_value = ties > 0 ? ties * weight(value, top, c, sh.table) : 0ULL;
    const float over = value == -INFINITY ? bottom : unordered(ordered(value) + 1);
    const Border s = search<true>(cluster, sh, row, over, top, top, c, [&](unsigned long long all) {
      const double want = ceil(static_cast<double>(top_p) * static_cast<double>(all + at_value));
      return want < 1.0 ? 1ULL : min(static_cast<unsigned long long>(want), all + at_value);
    });
    const unsigned long long w = weight(s.value == -INFINITY ? value : s.value, top, c, sh.table);
    const long long need = static_cast<long long>((s.target - s.above + w - 1) / w);
    ties = s.value == -INFINITY ? min(ties, need) : need;
    value = s.value == -INFINITY ? value : s.value;
  } else if (top_p < 1.f) {
    // All that is left has the largest logit.
    const double want = ceil(static_cast<double>(top_p) * static_cast<double>(ties));
    ties = min(ties, max(1LL, static_cast<long long>(want)));
  }
  const unsigned long long least =
      min_p > 0.f ? static_cast<unsigned long long>(ceil(fmin(static_cast<double>(min_p), 1.0) * kUnit)) : 0ULL;
  const unsigned long long w_tie = ties > 0 ? weight(value, top, c, sh.table) : 0ULL;
  if (w_tie < least) ties = 0;

  // The kept weights of every cell of 32 tokens, then of the CTA, then of the row.
  const int cells = (row.n + 31) / 32;
  for (int cell = warp; cell < cells; cell += kWarps) {
    const int i = cell * 32 + lane;
    const float z = i < row.n ? row.z[i] : -INFINITY;
    unsigned long long w = z > value ? weight(z, top, c, sh.table) : 0ULL;
    w = warp_sum(w >= least ? w : 0ULL);
    const int at = __popc(__ballot_sync(0xffffffffu, z == value && z > -INFINITY));
    if (lane == 0) sh.cell_over[cell] = w, sh.cell_ties[cell] = at;
  }
  __syncthreads();
  // A thread's two cells, and what lies ahead of them.
  static_assert(kCells == 2 * kThreads && kSampleMaxVocab <= kMaxCluster * kCells * 32, "cells");
  unsigned long long over[2], over_before;
  int at[2], at_before;
  {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int cell = 2 * static_cast<int>(threadIdx.x) + i;
      over[i] = cell < cells ? sh.cell_over[cell] : 0ULL;
      at[i] = cell < cells ? sh.cell_ties[cell] : 0;
    }
    const unsigned long long s = warp_scan(over[0] + over[1]);
    const int t = warp_scan(at[0] + at[1]);
    if (lane == 31) sh.warp_sum[warp] = s, sh.warp_ties[warp] = t;
    __syncthreads();
    over_before = s - over[0] - over[1];
    at_before = t - at[0] - at[1];
    unsigned long long all = 0;
    int all_at = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      over_before += w < warp ? sh.warp_sum[w] : 0ULL;
      at_before += w < warp ? sh.warp_ties[w] : 0;
      all += sh.warp_sum[w];
      all_at += sh.warp_ties[w];
    }
    if (threadIdx.x == 0) sh.over = all, sh.ties = all_at, sh.cell = -1;
  }
  cluster.sync();
  unsigned long long whole = 0, ahead = 0;
  long long ties_left = ties;  // for this CTA and those behind it
  {
    long long left = ties;
    for (int r = 0; r < ctas; ++r) {
      const Shared* other = cluster.map_shared_rank(&sh, r);
      if (r == rank) ahead = whole, ties_left = left;
      const long long take = min(left, static_cast<long long>(other->ties));
      whole += other->over + static_cast<unsigned long long>(take) * w_tie;
      left -= take;
    }
  }
  const float u = __ldg(p.uniform + b);
  unsigned long long target = 0;  // the token's running sum is the first over it
  if (u >= 1.f) target = whole - 1;
  else if (u > 0.f) target = min(static_cast<unsigned long long>(u * static_cast<double>(whole)), whole - 1);
  const auto kept = [](long long left, int n) {
    return static_cast<unsigned long long>(min(left, static_cast<long long>(n)));
  };
  // The cell, in this CTA or another; then, by its warp, the token.
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned long long from = ahead + over_before + kept(ties_left, at_before) * w_tie;
    over_before += over[i];
    at_before += at[i];
    const unsigned long long to = ahead + over_before + kept(ties_left, at_before) * w_tie;
    if (from <= target && target < to) {
      sh.cell = 2 * static_cast<int>(threadIdx.x) + i;
      sh.rest = target - from;
      sh.ties_before = at_before - at[i];
    }
  }
  cluster.sync();  // also: all have read the others' sums
  const int cell = sh.cell;
  if (cell < 0 || cell % kWarps != warp) return;
  const unsigned long long rest = sh.rest;
  ties_left -= min(ties_left, static_cast<long long>(sh.ties_before));
  const int i = cell * 32 + lane;
  const float z = i < row.n ? row.z[i] : -INFINITY;
  const bool tie = z == value && z > -INFINITY;
  unsigned long long w = z > value ? weight(z, top, c, sh.table) : 0ULL;
  if (w < least) w = 0;
  const int rank_at = __popc(__ballot_sync(0xffffffffu, tie) & ((1u << lane) - 1));
  if (tie && rank_at < ties_left) w = w_tie;
  const unsigned long long upto = warp_scan(w);
  if (upto - w <= rest && rest < upto) {
    p.tokens[b] = first + i;
    if (p.prob != nullptr) p.prob[b] = static_cast<float>(static_cast<double>(w) / static_cast<double>(whole));
  }
}

template <typename T, int VEC>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream) {
  // CTAs of a row: enough for at most 16384 values each (32768 in the longest
  // rows), and more where the rows alone would not fill the GPU.
  int ctas = 1;
  while (ctas < kMaxCluster && (a.V > ctas * 16384 || (a.B * ctas < 152 && a.V > ctas * kThreads * 4))) ctas *= 2;
  const int stretch = ((a.V + ctas - 1) / ctas + 31) / 32 * 32;
  const size_t smem = sizeof(Shared) + static_cast<size_t>(stretch) * sizeof(float);
  auto kernel = sample_kernel<T, VEC>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, a.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, stretch);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream) {
  const int vec = a.bf16 ? 8 : 4;
  const bool on16 = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.V % vec == 0 &&
                    (a.row_stride % vec == 0 || a.B == 1);
  if (a.bf16) return on16 ? launch<__nv_bfloat16, 8>(a, stream) : launch<__nv_bfloat16, 1>(a, stream);
  return on16 ? launch<float, 4>(a, stream) : launch<float, 1>(a, stream);
}

}  // namespace txl
