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
constexpr int kFew = 256;        // tokens that are compared each with each
constexpr int kMaxCluster = 8;
constexpr int kTable = 512;      // steps of the powers' table
constexpr int kOne = 44;         // the largest weight is 2^kOne
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
// (In fp64 this alone would take a microsecond.)
__device__ __forceinline__ Scale scale_of(float temperature) {
  constexpr float kHi = 1.442695041f, kLo = static_cast<float>(1.4426950408889634 - static_cast<double>(kHi));
  const float hi = kHi / temperature;
  if (!(hi > 0.f) || hi > FLT_MAX) return Scale{fminf(hi, FLT_MAX), 0.f};
  return Scale{hi, (fmaf(-hi, temperature, kHi) + kLo) / temperature};
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

constexpr int kGroup = 32, kGroups = kBins / kGroup;  // bins that are first looked at together
static_assert(kGroups == 64 && kThreads == 8 * kGroups, "eight threads a group");

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

struct Shared {
  unsigned long long table[kTable];
  union {
    unsigned long long bins[kBins];  // of the range at hand: sums of weights, or counts
    struct {                         // at the end: of cells of 32 tokens
      unsigned long long over[kCells];
      int ties[kCells];
    } cells;
  };
  unsigned long long groups[kMaxCluster][kGroups];
  uint4 ends[kMaxCluster];  // ordered: the smallest logit, the largest, a bound (below); how many
  Found found[kMaxCluster];
  Kept kept[kMaxCluster];
  float seg_z[kMaxCluster][kFew];
  int seg_i[kMaxCluster][kFew];
  float cand[kFew];
  int cand_i[kFew];
  unsigned long long cand_w[kFew];
  unsigned long long warp_sum[kWarps];
  int warp_ties[kWarps];
  uint32_t lo, hi, cut;  // of this CTA
  int live, n;
  int bin;                   // where the border lies,
  unsigned long long above;  // and the sum ahead of it
  float value;
  unsigned long long value_above;
  int cell;
  unsigned long long rest;
  int ties_before;
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

// The CTA's stretch of a row, in shared memory: -inf in place of NaN, the
// largest float of +inf, 0 of -0.
struct Row {
  float* z;
  int n, first;
};

// A thread's smallest and largest logit, ordered, and how many it has.
struct Ends {
  uint32_t lo = 0xffffffffu, hi = 0;
  int n = 0;
  __device__ __forceinline__ void take(float z) {
    if (z == -INFINITY) return;
    lo = min(lo, ordered(z));
    hi = max(hi, ordered(z));
    ++n;
  }
};

template <typename T, int VEC>
__device__ __forceinline__ Ends load_row(const Row& row, const T* from) {
  Ends ends;
  const auto clean = [](float x) { return isnan(x) ? -INFINITY : fminf(x + 0.f, FLT_MAX); };
  if constexpr (VEC == 1) {
#pragma unroll 8
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
      float x;
      if constexpr (sizeof(T) == 2) x = clean(__bfloat162float(from[i]));
      else x = clean(from[i]);
      row.z[i] = x;
      ends.take(x);
    }
  } else {
    static_assert(VEC * sizeof(T) == 16, "16 bytes");
#pragma unroll 4
    for (int i = threadIdx.x * VEC; i < row.n; i += kThreads * VEC) {  // row.n is a multiple of VEC
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(from + i));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float x[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if constexpr (sizeof(T) == 2) x[e] = clean(e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]));
        else x[e] = clean(__uint_as_float(w[e]));
        ends.take(x[e]);
      }
#pragma unroll
      for (int e = 0; e < VEC; e += 4)
        *reinterpret_cast<float4*>(row.z + i + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
  }
  return ends;
}

// A border's candidates, brought together from the CTAs' lists: thread i has the
// i-th, sh.cand and sh.cand_i have all.
template <int CTAS>
__device__ __forceinline__ void collect(Shared& sh, int n) {
  int i = threadIdx.x;
  if (i < n) {
    int r = 0;
    for (; r < CTAS - 1 && i >= sh.found[r].n; ++r) i -= sh.found[r].n;
    sh.cand[threadIdx.x] = sh.seg_z[r][i];
    sh.cand_i[threadIdx.x] = sh.seg_i[r][i];
  }
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

// The border of the sum of 1 (WEIGHTED false) or of the weights over the row's
// tokens with lo <= z <= hi, by falling z.  target_of(whole sum) gives the
// target, at least 1; where it is past the whole sum the border's value is
// -inf.  All threads of the cluster find the same.  Counts whose tokens down to
// the border are few end as a list.
template <bool WEIGHTED, int CTAS, typename F>
__device__ __forceinline__ Border search(cg::cluster_group& cluster, Shared& sh, const Row& row, float lo, float hi,
                                         float top, Scale c, F target_of) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = static_cast<int>(cluster.block_rank());
  unsigned long long above = 0, target = 0;
  Range range;
  for (int level = 0;; ++level) {
    range.set(lo, hi, level >= 2);
    for (int i = threadIdx.x; i < kBins / 2; i += kThreads)
      *reinterpret_cast<uint4*>(&sh.bins[2 * i]) = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) sh.n = 0, sh.lo = 0xffffffffu, sh.hi = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
      const float z = row.z[i];
      if (!range.has(z)) continue;
      if constexpr (WEIGHTED) {
        const unsigned long long w = weight(z, top, c, sh.table);
        if (w != 0) add64(&sh.bins[range.bin(z)], w);
      } else {
        atomicAdd(reinterpret_cast<unsigned int*>(&sh.bins[range.bin(z)]), 1u);
      }
    }
    __syncthreads();
    {  // the groups' sums, to all CTAs: of a group's eight threads each tells one
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&sh.bins[4 * threadIdx.x]);
      const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(&sh.bins[4 * threadIdx.x + 2]);
      unsigned long long sum = x.x + x.y + y.x + y.y;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int to = lane & 7;
      if (to < CTAS) cluster.map_shared_rank(&sh, to)->groups[rank][threadIdx.x >> 3] = sum;
    }
    cluster.sync();
    // Every warp finds the border's group; the first one then its bin.
    unsigned long long g[2] = {0, 0};
#pragma unroll
    for (int r = 0; r < CTAS; ++r) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&sh.groups[r][2 * lane]);
      g[0] += v.x;
      g[1] += v.y;
    }
    const unsigned long long upto = above + warp_scan(g[0] + g[1]);
    const unsigned long long all = __shfl_sync(0xffffffffu, upto, 31) - above;
    if (level == 0) {
      target = target_of(all);
      if (target > all) {
        cluster.sync();  // all have read the groups
        return Border{-INFINITY, all, target, 0};
      }
    }
    const int at_lane = __ffs(__ballot_sync(0xffffffffu, upto >= target)) - 1;
    const unsigned long long from = __shfl_sync(0xffffffffu, upto - g[0] - g[1], at_lane);
    const unsigned long long half = __shfl_sync(0xffffffffu, g[0], at_lane);
    const bool second = from + half < target;
    const int group = 2 * at_lane + second;
    if (warp == 0) {
      const unsigned long long before = from + (second ? half : 0ULL);
      unsigned long long b = 0, part[CTAS];
#pragma unroll
      for (int r = 0; r < CTAS; ++r) part[r] = cluster.map_shared_rank(sh.bins, r)[group * kGroup + lane];
#pragma unroll
      for (int r = 0; r < CTAS; ++r) b += part[r];
      const unsigned long long s = before + warp_scan(b);
      const int at = __ffs(__ballot_sync(0xffffffffu, s >= target)) - 1;
      if (lane == at) sh.bin = group * kGroup + lane, sh.above = s - b, sh.rest = b;
    }
    __syncthreads();
    const int bin = sh.bin;
    above = sh.above;
    // All tokens down to the border where they are few (counts), else the bin's;
    // and the bin's ends.
    const bool list = !WEIGHTED && level == 0 && above + sh.rest <= kFew;
    uint32_t l = 0xffffffffu, h = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
      const float z = row.z[i];
      if (!range.has(z)) continue;
      const int mine = range.bin(z);
      if (mine > bin || (mine < bin && !list)) continue;
      l = min(l, ordered(z));
      h = max(h, ordered(z));
      const int at = atomicAdd(&sh.n, 1);
      if (at >= kFew) continue;
      if (list) {
        Shared* to = cluster.map_shared_rank(&sh, 0);
        to->seg_z[rank][at] = z;
        to->seg_i[rank][at] = row.first + i;
      } else {
#pragma unroll
        for (int r = 0; r < CTAS; ++r) cluster.map_shared_rank(&sh, r)->seg_z[rank][at] = z;
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
    l = 0xffffffffu, h = 0;
#pragma unroll
    for (int r = 0; r < CTAS; ++r) {
      const Found f = sh.found[r];
      l = min(l, f.lo);
      h = max(h, f.hi);
      n += f.n;
    }
    if (list) {
      if (rank == 0) collect<CTAS>(sh, n);
      return Border{0.f, 0, target, n};
    }
    lo = unordered(l), hi = unordered(h);
    if (l == h) return Border{hi, above, target, 0};
    if (n > kFew) continue;
    collect<CTAS>(sh, n);
    if (static_cast<int>(threadIdx.x) < n)
      sh.cand_w[threadIdx.x] = WEIGHTED ? weight(sh.cand[threadIdx.x], top, c, sh.table) : 1ULL;
    __syncthreads();
    // Two threads for each of them: what lies above it, what equals it.
    static_assert(2 * kFew <= kThreads, "two threads a candidate");
    const float mine = sh.cand[min(static_cast<int>(threadIdx.x >> 1), n - 1)];
    unsigned long long over = 0, same = 0;
    for (int i = threadIdx.x & 1; i < n; i += 2) {
      const unsigned long long w = sh.cand_w[i];
      over += sh.cand[i] > mine ? w : 0ULL;
      same += sh.cand[i] == mine ? w : 0ULL;
    }
    over += above + __shfl_xor_sync(0xffffffffu, over, 1);
    same += __shfl_xor_sync(0xffffffffu, same, 1);
    if (over < target && target <= over + same) sh.value = mine, sh.value_above = over;  // by all its equals alike
    __syncthreads();
    return Border{sh.value, sh.value_above, target, 0};
  }
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

// The token of one of n <= kFew candidates, by one CTA: their places by falling
// logit and by index, then the filters and the draw on sums in those orders.
__device__ __forceinline__ void finish_list(Shared& sh, int n, const Settings& set, float top, Scale c,
                                            const SampleArgs& p, int b) {
  const int t = static_cast<int>(threadIdx.x), mine = t >> 1;
  const float z = sh.cand[min(mine, n - 1)];
  const int index = sh.cand_i[min(mine, n - 1)];
  int by_z = 0, by_i = 0;  // how many come first
  for (int i = t & 1; i < n; i += 2) {
    const bool lower = sh.cand_i[i] < index;
    by_z += sh.cand[i] > z || (sh.cand[i] == z && lower);
    by_i += lower;
  }
  by_z += __shfl_xor_sync(0xffffffffu, by_z, 1);
  by_i += __shfl_xor_sync(0xffffffffu, by_i, 1);
  const bool is = mine < n && (t & 1) == 0;
  const unsigned long long w = is && by_z < set.top_k ? weight(z, top, c, sh.table) : 0ULL;
  unsigned long long* sorted = sh.bins;  // the bins have served
  for (int i = t; i < 2 * kFew; i += kThreads) sorted[i] = 0;
  __syncthreads();
  if (is) sorted[by_z] = w;
  __syncthreads();
  unsigned long long all;
  const unsigned long long x = t < kFew ? sorted[t] : 0ULL;
  const unsigned long long before = block_scan(sh, x, &all);
  const unsigned long long target =
      set.top_p < 1.f ? (set.top_p > 0.f ? max(1ULL, share_of(set.top_p, all, true)) : 1ULL) : all;
  if (t < kFew) sorted[t] = before < target && x >= set.least ? x : 0ULL;
  __syncthreads();
  if (is) {
    sorted[kFew + by_i] = sorted[by_z];
    sh.cand_w[by_i] = static_cast<unsigned long long>(index);
  }
  __syncthreads();
  unsigned long long whole;
  const unsigned long long y = t < kFew ? sorted[kFew + t] : 0ULL;
  const unsigned long long from = block_scan(sh, y, &whole);
  const unsigned long long at = drawn(set.u, whole);
  if (from <= at && at < from + y) put(p, b, static_cast<int>(sh.cand_w[t]), y, whole);
}

template <typename T, int VEC, int CTAS>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs p, int stretch) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = static_cast<int>(blockIdx.y);
  const int first = rank * stretch;
  const Row row{reinterpret_cast<float*>(smem + sizeof(Shared)), max(0, min(stretch, p.V - first)), first};
  if (threadIdx.x == 0) sh.lo = 0xffffffffu, sh.hi = 0, sh.cut = 0xffffffffu, sh.live = 0, sh.cell = -1;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch_dependents();
  const float temperature = p.temperature != nullptr ? __ldg(p.temperature + b) : 1.f;
  const int k_asked = p.top_k != nullptr ? __ldg(p.top_k + b) : 0;
  const float p_asked = p.top_p != nullptr ? __ldg(p.top_p + b) : 1.f;
  const float m_asked = p.min_p != nullptr ? __ldg(p.min_p + b) : 0.f;
  Settings set;
  set.u = __ldg(p.uniform + b);
  for (int i = threadIdx.x; i < kTable; i += kThreads) sh.table[i] = kPowers.v[i];
  Ends mine = load_row<T, VEC>(row, static_cast<const T*>(p.logits) + b * p.row_stride + first);
  const bool greedy = !(temperature > 0.f);
  set.top_k = greedy ? 1 : k_asked;
  set.top_p = !greedy && p_asked < 1.f ? p_asked : 1.f;
  set.least = !greedy && m_asked > 0.f ? __float2ull_ru(fminf(m_asked, 1.f) * 0x1p44f) : 0ULL;
  const Scale c = greedy ? Scale{0.f, 0.f} : scale_of(temperature);

  // The row's largest and smallest logit, how many it has.  And a logit that is
  // not over the top_k-th largest, without which the search would put the whole
  // row into bins: of `parts` parts of the row, at least top_k, the smallest of
  // their largest.
  {
    int o = 32;  // threads of a part
    while (o > 1 && CTAS * kThreads / o < set.top_k) o >>= 1;
    uint32_t cut = mine.hi;
    for (int x = 1; x < o; x <<= 1) cut = max(cut, __shfl_xor_sync(0xffffffffu, cut, x));
    cut = __reduce_min_sync(0xffffffffu, cut);
    if (CTAS * kThreads < set.top_k) cut = 0;
    const uint32_t l = __reduce_min_sync(0xffffffffu, mine.lo), h = __reduce_max_sync(0xffffffffu, mine.hi);
    const int n = __reduce_add_sync(0xffffffffu, mine.n);
    if (lane == 0) {
      atomicMin(&sh.lo, l);
      atomicMax(&sh.hi, h);
      atomicMin(&sh.cut, cut);
      atomicAdd(&sh.live, n);
    }
  }
  __syncthreads();
  if (threadIdx.x < CTAS)
    cluster.map_shared_rank(&sh, threadIdx.x)->ends[rank] =
        make_uint4(sh.lo, sh.hi, sh.cut, static_cast<unsigned>(sh.live));
  cluster.sync();
  uint32_t l = 0xffffffffu, h = 0, cut = 0xffffffffu;
  int live = 0;
#pragma unroll
  for (int r = 0; r < CTAS; ++r) {
    const uint4 e = sh.ends[r];
    l = min(l, e.x);
    h = max(h, e.y);
    cut = min(cut, e.z);
    live += static_cast<int>(e.w);
  }
  if (live == 0) {
    if (rank == 0 && threadIdx.x == 0) put(p, b, -1, 0, 0);
    return;  // the whole cluster
  }
  const float top = unordered(h), bottom = unordered(l);

  // The threshold: tokens over `value`, and the first `ties` of those at it.
  float value = -INFINITY;
  long long ties = 0;
  if (set.top_k == 1) {
    value = top, ties = 1;
  } else if (set.top_k > 0 && set.top_k < live) {
    const auto target_of = [&](unsigned long long) { return static_cast<unsigned long long>(set.top_k); };
    const Border k = search<false, CTAS>(cluster, sh, row, unordered(max(l, cut)), top, top, c, target_of);
    if (k.list > 0) {
      if (rank == 0) finish_list(sh, k.list, set, top, c, p, b);
      return;
    }
    value = k.value;
    ties = static_cast<long long>(k.target - k.above);
  }
  if (set.top_p < 1.f) {
    // The smallest part of what is left that makes up top_p of it.
    const unsigned long long at_value = ties > 0 ? ties * weight(value, top, c, sh.table) : 0ULL;
    const auto target_of = [&](unsigned long long all) {
      return set.top_p > 0.f ? max(1ULL, share_of(set.top_p, all + at_value, true)) : 1ULL;
    };
    unsigned long long above = 0, target;
    float at = -INFINITY;
    if (value < top) {
      const Border s = search<true, CTAS>(cluster, sh, row, value == -INFINITY ? bottom : unordered(ordered(value) + 1),
                                          top, top, c, target_of);
      at = s.value, above = s.above, target = s.target;
    } else {
      target = target_of(0);
    }
    // (Rounded up; none of the weights that the sums count is 0.)
    const unsigned long long w = weight(at == -INFINITY ? value : at, top, c, sh.table);
    const long long need = static_cast<long long>((target - above + w - 1) / w);
    ties = at == -INFINITY ? min(ties, need) : need;
    value = at == -INFINITY ? value : at;
  }
  const unsigned long long w_tie = ties > 0 ? weight(value, top, c, sh.table) : 0ULL;
  if (w_tie < set.least) ties = 0;

  // The kept weights of every cell of 32 tokens, then of the CTA, then of the row.
  const int cells = (row.n + 31) / 32;
  for (int cell = warp; cell < cells; cell += kWarps) {
    const int i = cell * 32 + lane;
    const float z = i < row.n ? row.z[i] : -INFINITY;
    unsigned long long w = z > value ? weight(z, top, c, sh.table) : 0ULL;
    if (w < set.least) w = 0;
    if (__any_sync(0xffffffffu, w != 0)) w = warp_sum(w);
    const int at = __popc(__ballot_sync(0xffffffffu, z == value && z > -INFINITY));
    if (lane == 0) sh.cells.over[cell] = w, sh.cells.ties[cell] = at;
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
      over[i] = cell < cells ? sh.cells.over[cell] : 0ULL;
      at[i] = cell < cells ? sh.cells.ties[cell] : 0;
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
    if (threadIdx.x < CTAS) cluster.map_shared_rank(&sh, threadIdx.x)->kept[rank] = Kept{all, all_at};
  }
  cluster.sync();  // the last: nobody writes to another CTA from here on
  const auto kept = [](long long left, int n) {
    return static_cast<unsigned long long>(min(left, static_cast<long long>(n)));
  };
  unsigned long long whole = 0, ahead = 0;
  long long ties_left = 0;  // for this CTA and those behind it
  {
    long long left = ties;
#pragma unroll
    for (int r = 0; r < CTAS; ++r) {
      const Kept other = sh.kept[r];
      if (r == rank) ahead = whole, ties_left = left;
      const unsigned long long take = kept(left, other.ties);
      whole += other.over + take * w_tie;
      left -= static_cast<long long>(take);
    }
  }
  const unsigned long long target = drawn(set.u, whole);  // the token's running sum is the first over it
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
  __syncthreads();
  const int cell = sh.cell;
  if (cell < 0 || cell % kWarps != warp) return;
  const unsigned long long rest = sh.rest;
  ties_left -= min(ties_left, static_cast<long long>(sh.ties_before));
  const int i = cell * 32 + lane;
  const float z = i < row.n ? row.z[i] : -INFINITY;
  const bool tie = z == value && z > -INFINITY;
  unsigned long long w = z > value ? weight(z, top, c, sh.table) : 0ULL;
  if (w < set.least) w = 0;
  const int rank_at = __popc(__ballot_sync(0xffffffffu, tie) & ((1u << lane) - 1));
  if (tie && rank_at < ties_left) w = w_tie;
  const unsigned long long upto = warp_scan(w);
  if (upto - w <= rest && rest < upto) put(p, b, first + i, w, whole);
}

template <typename T, int VEC, int CTAS>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream) {
  const int stretch = ((a.V + CTAS - 1) / CTAS + 31) / 32 * 32;
  const size_t smem = sizeof(Shared) + static_cast<size_t>(stretch) * sizeof(float);
  auto kernel = sample_kernel<T, VEC, CTAS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
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
  // CTAs of a row: enough for at most 16384 values each (32768 in the longest
  // rows), and more where the rows alone would not fill the GPU.
  int ctas = 1;
  while (ctas < kMaxCluster && (a.V > ctas * 16384 || (a.B * ctas < 152 && a.V > ctas * kThreads * 4))) ctas *= 2;
  switch (ctas) {
    case 1: return launch<T, VEC, 1>(a, stream);
    case 2: return launch<T, VEC, 2>(a, stream);
    case 4: return launch<T, VEC, 4>(a, stream);
    default: return launch<T, VEC, 8>(a, stream);
  }
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
