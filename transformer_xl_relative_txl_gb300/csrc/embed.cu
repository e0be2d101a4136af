// Token ids to rows of an embedding table, and the table's gradient.
//
//   out[t] = scale * table[token[t]]
//   dtable[v] (+)= scale * sum of dout[t] over the t with token[t] == v
//
// A token outside 0 .. V-1 is padding: zeros, and no part of any sum.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "pdl.cuh"
#include "tokens.h"
#include "txl_device.cuh"

namespace txl {
namespace {

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// N consecutive values of a row in fp32, and back with one rounding.
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  if constexpr (N == 1) {
    if constexpr (sizeof(T) == 2) v[0] = __bfloat162float(*p);
    else v[0] = *p;
  } else if constexpr (sizeof(T) == 2) {
    uint32_t w[N / 2];
    if constexpr (N == 8) *reinterpret_cast<uint4*>(w) = __ldg(reinterpret_cast<const uint4*>(p));
    else *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(p));
#pragma unroll
    for (int e = 0; e < N / 2; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p + e));
      v[e] = x.x, v[e + 1] = x.y, v[e + 2] = x.z, v[e + 3] = x.w;
    }
  }
}

template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    if constexpr (sizeof(T) == 2) *p = __float2bfloat16(v[0]);
    else *p = v[0];
  } else if constexpr (sizeof(T) == 2) {
    static_assert(N == 8, "eight values");
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4)
      *reinterpret_cast<float4*>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
}

constexpr int kLookupThreads = 256;

// 2^lanes_log threads go along a row, 8 columns each at a time (N = 1: one,
// where rows do not start on 16 bytes); a thread takes U rows at once, so that
// their loads are in flight together.  Bound by memory: 11264 rows of 512, fp32 to
// bf16, take 4.0 us with ids by frequency, 20 MB at three quarters of a copy's
// rate; 64 rows 2.1, the launch.
template <typename TI, typename TO, int N, int U>
__global__ void __launch_bounds__(kLookupThreads)
    embed_forward_kernel(const int* __restrict__ tokens, const TI* __restrict__ table, TO* __restrict__ out, int T,
                         int V, int d, int lanes_log, float scale) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int lane = threadIdx.x & ((1 << lanes_log) - 1);
  const int rows = kLookupThreads >> lanes_log;  // of a pass
  const long long t0 = static_cast<long long>(blockIdx.x) * rows * U + (threadIdx.x >> lanes_log);
  int id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long t = t0 + static_cast<long long>(u) * rows;
    id[u] = t < T ? __ldg(tokens + t) : -1;
    if (id[u] >= V) id[u] = -1;
  }
  for (int c = lane * N; c < d; c += N << lanes_log) {
    float v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (id[u] >= 0) {
        load_n<TI, N>(table + static_cast<size_t>(id[u]) * d + c, v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[u][e] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = t0 + static_cast<long long>(u) * rows;
      if (t >= T) continue;
      if (id[u] >= 0) {  // (0 * scale would not be 0 for an infinite scale)
#pragma unroll
        for (int e = 0; e < N; ++e) v[u][e] *= scale;
      }
      store_n<TO, N>(out + static_cast<size_t>(t) * d + c, v[u]);
    }
  }
}

template <typename TI, typename TO, int N>
cudaError_t forward_typed(const int* tokens, const void* table, void* out, int T, int V, int d, float scale,
                          cudaStream_t stream) {
  const int vecs = (d + N - 1) / N;
  int lanes_log = 0;
  while ((1 << lanes_log) < vecs && (1 << lanes_log) < kLookupThreads) ++lanes_log;
  const int rows = kLookupThreads >> lanes_log;
  const auto go = [&](auto kernel, int u) {
    const int per = rows * u;
    return launch_dependent(kernel, dim3((T + per - 1) / per), dim3(kLookupThreads), 0, stream, tokens,
                            static_cast<const TI*>(table), static_cast<TO*>(out), T, V, d, lanes_log, scale);
  };
  // Four rows a thread once that still leaves a block for each of 4 x 152 places:
  // 16384 rows of 512 (rows anywhere in the table) take 7.8 us by four and 8.5 by
  // one, 2500 of 1024 3.3 and 3.0, 64 of 512 1.7 and 1.6.
  if (T / (4 * rows) >= 608) return go(embed_forward_kernel<TI, TO, N, 4>, 4);
  return go(embed_forward_kernel<TI, TO, N, 1>, 1);
}

// Rows of 16-byte vectors, or elements one by one: 11264 rows (anywhere) of 300 in
// bf16 take 6.2 us, of 304 3.8, of which the bytes need 2.0; from fp32 7.5 and 5.1;
// of 512 from fp32 9.4 where out starts off 16 bytes and 6.9 on them.
bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename TI, typename TO>
cudaError_t forward_any(const int* tokens, const void* table, void* out, int T, int V, int d, float scale,
                        cudaStream_t stream) {
  if (d % 8 == 0 && on16(table) && on16(out))
    return forward_typed<TI, TO, 8>(tokens, table, out, T, V, d, scale, stream);
  return forward_typed<TI, TO, 1>(tokens, table, out, T, V, d, scale, stream);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// One kernel, in which every CTA owns some rows of the table, of which it
// writes COLS columns: the rows v with v % classes == its class, so that the
// common ids, which vocabularies number first, are spread over all CTAs.  It
// reads all ids, keeps its own in the order of their places, sorts them by row
// and place and sums each row's gradients, in shares that are equal whatever the
// rows' lengths.  A row's sum has one order, which the ids, V and d decide, and is
// put into the table once a pass: added to it, by one atomic whose result nothing
// waits for, or stored.  A pass takes up to 32768 ids, of which a CTA's own must fit
// its lists: where a row has most of them, a half, a quarter or an eighth of that,
// and each length tried reads its ids again, in every pass (of 11264 equal ids 47168
// are read).
//
// The gradients' rows are asked for as soon as the ids are listed, so that they
// are on their way to L2 while the list is sorted and the other rows zeroed.
//
// No kernel ahead of it and no workspace: adding by atomics as the ids come needs
// neither but has no order; sorting in a kernel of its own takes two launches more.
// The price is that every CTA reads all ids.  11264 ids by frequency of 32768 rows,
// d = 512 in bf16, the table written whole: 25.6 us, of which the bytes (79 MB) need
// 11.6; added to a table 18.4, of 4.2.  A chain of steps, each short: at 2 CTAs an
// SM the schedulers issue half of the time, shared memory's and the barriers'
// latencies the rest.  A row with a large part of all ids is summed by one CTA a
// slice: 11264 equal ids take 107 us (table written whole: 119), 4096 35.
constexpr int kGradThreads = 512, kGradWarps = kGradThreads / 32;
constexpr int kMaxLocal = 16384;  // rows of a CTA
constexpr int kPlaceBits = 15;
constexpr int kChunk = 1 << kPlaceBits;  // ids at a time
constexpr int kList = 4096;       // of them a CTA's own
constexpr int kWarpList = kList / kGradWarps;
constexpr int kAhead = 4;         // gradient rows of a worker; as many again in flight
constexpr uint32_t kNone = 0xffffffffu;
static_assert(kMaxLocal <= 1 << (32 - kPlaceBits - 1), "an entry, row and place, fits 31 bits");

struct GradSmem {  // ahead of end[local rows]
  uint32_t list[kList];  // by warp; then the ranks of the next's
  uint32_t line[kList];  // all, by place
  uint32_t sorted[kList];
  alignas(16) float part[kGradThreads][2][4];
  int counts[kGradWarps];
  int sums[kGradWarps];
};

struct GradArgs {
  const int* tokens;
  const void* dout;
  float* dtable;
  int T, V, d;
  int classes;       // odd
  uint32_t inverse;  // of classes, modulo 2^32
  float scale;
  bool accumulate;
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A worker's columns of a row, COLS / 4 lanes: 4 a lane in a line (N = 4) or
// COLS / 4 apart (N = 1, where rows do not start on 16 bytes).
template <typename T, int N, int COLS>
struct Columns {
  static constexpr int kLanes = COLS / 4;
  int c0, left;  // the slice's first column, how many it has
  struct Raw {
    uint32_t w[N == 4 ? static_cast<int>(sizeof(T)) : 4];
  };
  __device__ __forceinline__ int at(int e) const {
    const int l = static_cast<int>(threadIdx.x) % kLanes;
    return N == 4 ? l * 4 + e : l + kLanes * e;
  }
  __device__ __forceinline__ void load(const T* row, Raw* r) const {
    if constexpr (N == 4 && sizeof(T) == 2) {
      if (at(0) < left) *reinterpret_cast<uint2*>(r->w) = __ldg(reinterpret_cast<const uint2*>(row + c0 + at(0)));
    } else if constexpr (N == 4) {
      if (at(0) < left) *reinterpret_cast<uint4*>(r->w) = __ldg(reinterpret_cast<const uint4*>(row + c0 + at(0)));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (at(e) >= left) continue;
        float x[1];
        load_n<T, 1>(row + c0 + at(e), x);
        r->w[e] = __float_as_uint(x[0]);
      }
    }
  }
  __device__ __forceinline__ void add(const Raw& r, float (&sum)[4]) const {
    if constexpr (N == 4 && sizeof(T) == 2) {
      sum[0] += bf16_lo(r.w[0]), sum[1] += bf16_hi(r.w[0]);
      sum[2] += bf16_lo(r.w[1]), sum[3] += bf16_hi(r.w[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += __uint_as_float(r.w[e]);
    }
  }
  // To what is there (a subnormal result becomes 0).
  __device__ __forceinline__ void add_to(float* row, const float (&v)[4]) const {
    if constexpr (N == 4) {
      if (at(0) < left)
        asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(row + c0 + at(0)), "f"(v[0]), "f"(v[1]),
                     "f"(v[2]), "f"(v[3])
                     : "memory");
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at(e) < left) atomicAdd(row + c0 + at(e), v[e]);
    }
  }
  __device__ __forceinline__ void store(float* row, const float (&v)[4]) const {
    if constexpr (N == 4) {
      if (at(0) < left) *reinterpret_cast<float4*>(row + c0 + at(0)) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at(e) < left) row[c0 + at(e)] = v[e];
    }
  }
};

template <typename T, int N, int COLS>
__global__ void __launch_bounds__(kGradThreads, 2) embed_backward_kernel(const GradArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  GradSmem& sh = *reinterpret_cast<GradSmem*>(smem);
  int* end = reinterpret_cast<int*>(smem + sizeof(GradSmem));  // of a local row's entries in `sorted`
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = static_cast<int>(blockIdx.x);
  const int rows = (p.V - mine + p.classes - 1) / p.classes;  // <= kMaxLocal
  using C = Columns<T, N, COLS>;
  constexpr int kWorkers = kGradThreads / C::kLanes;
  const int worker = static_cast<int>(threadIdx.x) / C::kLanes;
  C cols;
  cols.c0 = static_cast<int>(blockIdx.y) * COLS;
  cols.left = min(COLS, p.d - cols.c0);
  const T* dout = static_cast<const T*>(p.dout);
  grid_dep_wait();
  grid_dep_launch_dependents();

  long long base = 0;
  for (bool begun = false; !begun || base < p.T; begun = true) {  // (without ids: zeros)
    int n = static_cast<int>(min(static_cast<long long>(kChunk), p.T - base));
    const bool add = p.accumulate || begun;
    for (int i = threadIdx.x; i < rows; i += kGradThreads) end[i] = 0;
    int total, before;
    for (;;) {
      // The ids of this CTA's rows, in order: each warp lists those of its stretch.
      const int part = (n + kGradThreads - 1) / kGradThreads * 32;
      const int i0 = min(n, warp * part), i1 = min(n, i0 + part);
      uint32_t* list = sh.list + warp * kWarpList;
      int count = 0;
      constexpr int kRead = 16;  // ids of a lane on their way
      for (int i = i0; i < i1; i += kRead * 32) {
        int v[kRead];
#pragma unroll
        for (int u = 0; u < kRead; ++u) {
          const int at = i + u * 32 + lane;
          v[u] = at < i1 ? __ldg(p.tokens + base + at) : -1;
        }
#pragma unroll
        for (int u = 0; u < kRead; ++u) {
          if (i + u * 32 >= i1) break;
          // Of this class: v - mine a multiple of classes, q classes by 32-bit words,
          // and not one of those that wrap: q below the local rows (no padding is).
          const uint32_t q = (static_cast<uint32_t>(v[u]) - static_cast<uint32_t>(mine)) * p.inverse;
          const bool is = q < static_cast<uint32_t>(rows);
          const uint32_t b = __ballot_sync(0xffffffffu, is);
          const int at = count + __popc(b & ((1u << lane) - 1));
          if (is && at < kWarpList) list[at] = q << kPlaceBits | static_cast<uint32_t>(i + u * 32 + lane);
          count += __popc(b);
        }
      }
      if (lane == 0) sh.counts[warp] = count;
      __syncthreads();
      total = before = 0;
      bool fits = true;
#pragma unroll
      for (int w = 0; w < kGradWarps; ++w) {
        const int c = sh.counts[w];
        before += w < warp ? c : 0;
        total += c;
        fits = fits && c <= kWarpList;
      }
      if (fits) break;
      __syncthreads();
      n /= 2;  // many ids of this CTA in a row: fewer at a time (kList of them always fit)
    }
    // All in one line, counted by row; their rows on the way to L2.
    {
      const int count = sh.counts[warp];
      const uint32_t* list = sh.list + warp * kWarpList;
      constexpr int kBytes = COLS * static_cast<int>(sizeof(T)), kLines = (kBytes + 127) / 128;
      for (int i = lane; i < count * kLines; i += 32) {
        const int c = i % kLines * (128 / static_cast<int>(sizeof(T)));
        if (c < cols.left) prefetch_l2(dout + (base + (list[i / kLines] & (kChunk - 1))) * p.d + cols.c0 + c);
      }
      for (int i = lane; i < count; i += 32) {
        const uint32_t e = list[i];
        sh.line[before + i] = e;
        atomicAdd(&end[e >> kPlaceBits], 1);
      }
    }
    __syncthreads();
    const long long first = base;
    base += n;
    // Rows without an id are zeros.
    if (!add) {
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      const size_t step = static_cast<size_t>(kWorkers) * p.classes * p.d;
      float* to = p.dtable + (static_cast<size_t>(worker) * p.classes + mine) * p.d;
#pragma unroll 4
      for (int i = worker; i < rows; i += kWorkers, to += step)
        if (end[i] == 0) cols.store(to, zero);
    }
    if (total == 0) {  // the same for all threads
      __syncthreads();
      continue;
    }
    if (!add) __syncthreads();
    {  // where each row's entries begin
      const int per = (rows + kGradThreads - 1) / kGradThreads;
      const int lo = min(rows, static_cast<int>(threadIdx.x) * per), hi = min(rows, lo + per);
      int x = 0;
      for (int i = lo; i < hi; ++i) x += end[i];
      int s = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      if (lane == 31) sh.sums[warp] = s;
      __syncthreads();
      int at = s - x;
#pragma unroll
      for (int w = 0; w < kGradWarps; ++w) at += w < warp ? sh.sums[w] : 0;
      for (int i = lo; i < hi; ++i) {
        const int c = end[i];
        end[i] = at;
        at += c;
      }
    }
    __syncthreads();
    // By row, and within a row by place.  All warps look, among 32 entries, how
    // many come ahead of one in its row, and how many there are; then the first warp
    // takes the 32 through the rows' counters, which move on to each row's end.
    uint32_t* ranks = sh.list;
    for (int i = warp * 32; i < total; i += kGradThreads) {
      const uint32_t row = i + lane < total ? sh.line[i + lane] >> kPlaceBits : kNone;
      const uint32_t same = __match_any_sync(0xffffffffu, row);
      ranks[i + lane] = __popc(same & ((1u << lane) - 1)) | static_cast<uint32_t>(__popc(same)) << 8;
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t e = lane < total ? sh.line[lane] : kNone, r = ranks[lane];
      for (int i = 0; i < total; i += 32) {
        const bool in = e != kNone;
        int* counter = end + (in ? e >> kPlaceBits : 0);
        const int at = in ? *counter : 0;
        __syncwarp();
        if (in && (r & 255) == 0) *counter = at + static_cast<int>(r >> 8);
        if (in) sh.sorted[at + static_cast<int>(r & 255)] = e;
        const int j = i + 32 + lane;
        e = j < total ? sh.line[j] : kNone;
        r = j < total ? ranks[j] : 0;
        __syncwarp();
      }
    }
    __syncthreads();
    // Equal shares of the entries.  A row that a share's border cuts is put
    // together from the workers' parts.
    const int per = (total + kWorkers - 1) / kWorkers;
    const int p0 = min(total, worker * per), p1 = min(total, p0 + per);
    const uint32_t row_before = p0 > 0 ? sh.sorted[p0 - 1] >> kPlaceBits : kNone;
    const uint32_t row_behind = p1 < total ? sh.sorted[p1] >> kPlaceBits : kNone;
    const auto put = [&](uint32_t row, const float (&sum)[4]) {
      const float v[4] = {sum[0] * p.scale, sum[1] * p.scale, sum[2] * p.scale, sum[3] * p.scale};
      float* to = p.dtable + (static_cast<size_t>(row) * p.classes + mine) * p.d;
      if (add) cols.add_to(to, v);
      else cols.store(to, v);
    };
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    typename C::Raw next[kAhead] = {};
    const T* from = dout + first * p.d;
    const auto read = [&](int q) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (q + u < p1) cols.load(from + static_cast<size_t>(sh.sorted[q + u] & (kChunk - 1)) * p.d, &next[u]);
    };
    read(p0);
    for (int q = p0; q < p1; q += kAhead) {
      typename C::Raw v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) v[u] = next[u];
      read(q + kAhead);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (q + u >= p1) break;
        cols.add(v[u], sum);
        const uint32_t row = sh.sorted[q + u] >> kPlaceBits;
        if (q + u + 1 < p1 && sh.sorted[q + u + 1] >> kPlaceBits == row) continue;
        const bool cut_before = row == row_before, cut_behind = q + u + 1 == p1 && row == row_behind;
        if (!cut_before && !cut_behind) {
          put(row, sum);
        } else {
          float* part = sh.part[threadIdx.x][!cut_before];  // 0: the end, or the middle, of an earlier worker's row
          *reinterpret_cast<float4*>(part) = make_float4(sum[0], sum[1], sum[2], sum[3]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[x] = 0.f;
      }
    }
    __syncthreads();
    if (p0 < p1 && row_behind != kNone) {  // a row that begins in this worker's share and ends in another's
      const uint32_t row = sh.sorted[p1 - 1] >> kPlaceBits;
      if (row == row_behind && row != row_before) {
        const int last = (end[row] - 1) / per;
        float4 x = *reinterpret_cast<const float4*>(sh.part[threadIdx.x][1]);
#pragma unroll 4
        for (int w = worker + 1; w <= last; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(sh.part[threadIdx.x + (w - worker) * C::kLanes][0]);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const float all[4] = {x.x, x.y, x.z, x.w};
        put(row, all);
      }
    }
    __syncthreads();
  }
}

template <typename T, int N, int COLS>
cudaError_t backward_sliced(GradArgs a, cudaStream_t stream) {
  const int slices = (a.d + COLS - 1) / COLS;
  // Two CTAs for each SM, and no more rows a CTA than it has room for; odd.
  a.classes = std::max((2 * 152 / slices - 1) | 1, ((a.V + kMaxLocal - 1) / kMaxLocal) | 1);
  a.classes = std::min(a.classes, (a.V - 1) | 1);
  a.inverse = 1;  // Newton's steps: each doubles the bits that are right
  for (int i = 0; i < 5; ++i) a.inverse *= 2 - static_cast<uint32_t>(a.classes) * a.inverse;
  const size_t smem = sizeof(GradSmem) + static_cast<size_t>((a.V + a.classes - 1) / a.classes) * sizeof(int);
  auto kernel = embed_backward_kernel<T, N, COLS>;
  // The most that any call needs: another thread may set it at the same time.
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       sizeof(GradSmem) + kMaxLocal * sizeof(int));
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(a.classes, slices), dim3(kGradThreads), smem, stream, a);
}

template <typename T, int N>
cudaError_t backward_typed(const GradArgs& a, cudaStream_t stream) {
  // Narrow slices share a common id's rows among more CTAs; wide ones leave each
  // CTA fewer ids to sort.  32 columns and 64, in us: d = 64 18.7 and 20.1, d = 333
  // 13.8 and 14.9, d = 512 25.9 and 25.7, d = 1024 24.5 and 16.4, d = 2048 78 and 44
  // (128: 17.1, 27.7, 16.9 and 45 from d = 333 on).
  if (a.d <= 400) return backward_sliced<T, N, 32>(a, stream);
  return backward_sliced<T, N, 64>(a, stream);
}

}  // namespace

cudaError_t launch_embed_forward(const int* tokens, const void* table, void* out, int T, int V, int d, float scale,
                                 bool table_bf16, bool out_bf16, cudaStream_t stream) {
  if (table_bf16 && out_bf16)
    return forward_any<__nv_bfloat16, __nv_bfloat16>(tokens, table, out, T, V, d, scale, stream);
  if (table_bf16) return forward_any<__nv_bfloat16, float>(tokens, table, out, T, V, d, scale, stream);
  if (out_bf16) return forward_any<float, __nv_bfloat16>(tokens, table, out, T, V, d, scale, stream);
  return forward_any<float, float>(tokens, table, out, T, V, d, scale, stream);
}

cudaError_t launch_embed_backward(const int* tokens, const void* dout, float* dtable, int T, int V, int d, float scale,
                                  bool accumulate, bool dout_bf16, cudaStream_t stream) {
  GradArgs a{tokens, dout, dtable, T, V, d, 0, 0, scale, accumulate};
  const bool vec = d % 4 == 0 && on16(dtable) && reinterpret_cast<uintptr_t>(dout) % (dout_bf16 ? 8 : 16) == 0;
  if (dout_bf16)
    return vec ? backward_typed<__nv_bfloat16, 4>(a, stream) : backward_typed<__nv_bfloat16, 1>(a, stream);
  return vec ? backward_typed<float, 4>(a, stream) : backward_typed<float, 1>(a, stream);
}

}  // namespace txl
