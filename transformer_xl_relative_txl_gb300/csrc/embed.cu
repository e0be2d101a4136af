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
// their loads are in flight together.
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
  // Four rows a thread once that still leaves a block for each of 4 x 152 places.
  if (T / (4 * rows) >= 608) return go(embed_forward_kernel<TI, TO, N, 4>, 4);
  return go(embed_forward_kernel<TI, TO, N, 1>, 1);
}

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
// writes kCols columns: the rows v with v % classes == its class, so that the
// common ids, which vocabularies number first, are spread over all CTAs.  It
// reads all ids, keeps its own in the order of their places, sorts them by row
// and sums each row's gradients, which its warps share equally whatever the
// rows' lengths.  Nothing is added by atomics: a row's sum has one order,
// which the ids alone decide.
constexpr int kGradThreads = 512, kGradWarps = kGradThreads / 32;
constexpr int kCols = 128;        // columns of a CTA
constexpr int kMaxLocal = 8192;   // rows of a CTA
constexpr int kChunk = 8192;      // ids at a time
constexpr int kRounds = kChunk / kGradThreads;
constexpr int kPlaceBits = 13;    // of a place in a chunk
constexpr int kAhead = 4;         // gradient rows in flight per warp
static_assert(kChunk <= 1 << kPlaceBits && kMaxLocal <= 1 << (32 - kPlaceBits), "an entry fits 32 bits");

struct GradSmem {  // ahead of first[local + 1], list[chunk], sorted[chunk]
  float part[kGradWarps][2][kCols];
  int counts[kRounds * kGradWarps];
  int sums[kGradWarps];
  int total;
};

struct GradArgs {
  const int* tokens;
  const void* dout;
  float* dtable;
  int T, V, d, classes;
  unsigned long long inverse;  // 2^40 / classes + 1
  float scale;
  bool accumulate;
  int local, chunk;  // the shared arrays' lengths
};

// Exclusive sum over the block, and the total.
__device__ __forceinline__ int block_scan(int x, int* sums, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kGradWarps; ++w) {
    const int y = sums[w];
    before += w < warp ? y : 0;
    all += y;
  }
  __syncthreads();
  *total = all;
  return before + s - x;
}

// A warp's columns of a row: 4 a lane in a line (N = 4) or every 32nd (N = 1,
// where rows do not start on 16 bytes).
template <int N>
struct Columns {
  int c0, left;  // the slice's first column, how many it has
  __device__ __forceinline__ int at(int e) const {
    return N == 4 ? (threadIdx.x & 31) * 4 + e : (threadIdx.x & 31) + 32 * e;
  }
  template <typename T>
  __device__ __forceinline__ void load(const T* row, float (&v)[4]) const {
    if constexpr (N == 4) {
      if (at(0) < left) load_n<T, 4>(row + c0 + at(0), v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at(e) < left) {
          float x[1];
          load_n<T, 1>(row + c0 + at(e), x);
          v[e] = x[0];
        }
    }
  }
  __device__ __forceinline__ void store(float* row, const float (&v)[4]) const {
    if constexpr (N == 4) {
      if (at(0) < left) store_n<float, 4>(row + c0 + at(0), v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at(e) < left) row[c0 + at(e)] = v[e];
    }
  }
};

template <typename T, int N>
__global__ void __launch_bounds__(kGradThreads, 2) embed_backward_kernel(const GradArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  GradSmem& sh = *reinterpret_cast<GradSmem*>(smem);
  int* first = reinterpret_cast<int*>(smem + sizeof(GradSmem));  // of each local row, in `sorted`
  uint32_t* list = reinterpret_cast<uint32_t*>(first + p.local + 1);
  uint32_t* sorted = list + p.chunk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = static_cast<int>(blockIdx.x);
  const int rows = (p.V - mine + p.classes - 1) / p.classes;  // <= p.local
  Columns<N> cols;
  cols.c0 = static_cast<int>(blockIdx.y) * kCols;
  cols.left = min(kCols, p.d - cols.c0);
  const T* dout = static_cast<const T*>(p.dout);
  grid_dep_wait();
  grid_dep_launch_dependents();

  for (long long base = 0; base == 0 || base < p.T; base += p.chunk) {  // (without ids: zeros)
    const int n = static_cast<int>(min(static_cast<long long>(p.chunk), p.T - base));
    const bool add = p.accumulate || base > 0;
    // The ids of this CTA's rows, in order.
    uint32_t entry[kRounds];
    uint32_t own = 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int i = r * kGradThreads + static_cast<int>(threadIdx.x);
      const int v = i < n ? __ldg(p.tokens + base + i) : -1;
      const uint32_t q = static_cast<uint32_t>(static_cast<uint32_t>(v) * p.inverse >> 40);  // v / classes, v < 2^24
      const bool is = v >= 0 && v < p.V && v - static_cast<int>(q) * p.classes == mine;
      entry[r] = q << kPlaceBits | static_cast<uint32_t>(i);
      const uint32_t b = __ballot_sync(0xffffffffu, is);
      own |= static_cast<uint32_t>(is) << r;
      if (lane == 0) sh.counts[r * kGradWarps + warp] = __popc(b);
    }
    for (int i = threadIdx.x; i <= rows; i += kGradThreads) first[i] = 0;
    __syncthreads();
    static_assert(kRounds * kGradWarps <= kGradThreads, "a count a thread");
    {
      int total;
      const int x = threadIdx.x < kRounds * kGradWarps ? sh.counts[threadIdx.x] : 0;
      const int before = block_scan(x, sh.sums, &total);
      if (threadIdx.x < kRounds * kGradWarps) sh.counts[threadIdx.x] = before;
      if (threadIdx.x == 0) sh.total = total;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const bool is = own >> r & 1;
      const uint32_t b = __ballot_sync(0xffffffffu, is);
      if (is) {
        list[sh.counts[r * kGradWarps + warp] + __popc(b & ((1u << lane) - 1))] = entry[r];
        atomicAdd(&first[entry[r] >> kPlaceBits], 1);
      }
    }
    __syncthreads();
    const int total = sh.total;
    // Rows without an id are zeros.  (Before the counts become places.)
    if (!add) {
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = warp; i < rows; i += kGradWarps)
        if (first[i] == 0) cols.store(p.dtable + (static_cast<size_t>(i) * p.classes + mine) * p.d, zero);
      __syncthreads();
    }
    if (total == 0) continue;  // the same for all threads
    {
      const int per = (rows + kGradThreads - 1) / kGradThreads;
      const int lo = min(rows, static_cast<int>(threadIdx.x) * per), hi = min(rows, lo + per);
      int x = 0;
      for (int i = lo; i < hi; ++i) x += first[i];
      int all;
      int at = block_scan(x, sh.sums, &all);
      for (int i = lo; i < hi; ++i) {
        const int c = first[i];
        first[i] = at;
        at += c;
      }
      if (threadIdx.x == 0) first[rows] = all;
    }
    __syncthreads();
    // By row, and within a row by place: one warp, 32 entries at a time.
    // `first` moves on to each row's end.
    if (warp == 0) {
      for (int i = 0; i < total; i += 32) {
        const bool in = i + lane < total;
        const uint32_t e = in ? list[i + lane] : 0xffffffffu;
        const uint32_t same = __match_any_sync(0xffffffffu, e >> kPlaceBits);
        const int rank = __popc(same & ((1u << lane) - 1));
        int at = 0;
        if (in && rank == 0) {
          at = first[e >> kPlaceBits];
          first[e >> kPlaceBits] = at + __popc(same);
        }
        at = __shfl_sync(0xffffffffu, at, __ffs(same) - 1);
        if (in) sorted[at + rank] = e;
        __syncwarp();
      }
    }
    __syncthreads();
    // Equal shares of the sorted entries.  A row that a share's border cuts is
    // put together from the warps' parts.  first[i] is now row i's end.
    const int per = (total + kGradWarps - 1) / kGradWarps;
    const int p0 = min(total, warp * per), p1 = min(total, p0 + per);
    const auto begin_of = [&](int i) { return i == 0 ? 0 : first[i - 1]; };
    const auto put = [&](int row, const float (&sum)[4], const float (&old)[4]) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = add ? fmaf(sum[e], p.scale, old[e]) : sum[e] * p.scale;
      cols.store(p.dtable + (static_cast<size_t>(row) * p.classes + mine) * p.d, v);
    };
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int q = p0; q < p1; q += kAhead) {
      float v[kAhead][4], old[kAhead][4];
      uint32_t e[kAhead + 1];
#pragma unroll
      for (int u = 0; u <= kAhead; ++u) e[u] = q + u < p1 ? sorted[q + u] : 0xffffffffu;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
#pragma unroll
        for (int x = 0; x < 4; ++x) v[u][x] = 0.f, old[u][x] = 0.f;
        if (q + u < p1) {
          cols.load(dout + (base + (e[u] & ((1u << kPlaceBits) - 1))) * p.d, v[u]);
          const int row = static_cast<int>(e[u] >> kPlaceBits);
          if (add && e[u + 1] >> kPlaceBits != e[u] >> kPlaceBits && first[row] <= p1 && begin_of(row) >= p0)
            cols.load(p.dtable + (static_cast<size_t>(row) * p.classes + mine) * p.d, old[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (q + u >= p1) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[x] += v[u][x];
        if (e[u + 1] >> kPlaceBits == e[u] >> kPlaceBits) continue;
        const int row = static_cast<int>(e[u] >> kPlaceBits);
        const bool from_here = begin_of(row) >= p0;
        if (from_here && first[row] <= p1) {
          put(row, sum, old[u]);
        } else {
          float* part = sh.part[warp][from_here];
#pragma unroll
          for (int x = 0; x < 4; ++x) part[lane + 32 * x] = sum[x];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[x] = 0.f;
      }
    }
    __syncthreads();
    if (p0 < p1) {  // a row that begins in this warp's share and ends in another's
      const int row = static_cast<int>(sorted[p1 - 1] >> kPlaceBits);
      if (begin_of(row) >= p0 && first[row] > p1) {
        float old[4] = {0.f, 0.f, 0.f, 0.f};
        if (add) cols.load(p.dtable + (static_cast<size_t>(row) * p.classes + mine) * p.d, old);
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[x] = sh.part[warp][1][lane + 32 * x];
        for (int w = warp + 1; w < kGradWarps && w * per < first[row]; ++w)
#pragma unroll
          for (int x = 0; x < 4; ++x) sum[x] += sh.part[w][0][lane + 32 * x];
        put(row, sum, old);
      }
    }
    __syncthreads();
  }
}

template <typename T, int N>
cudaError_t backward_typed(GradArgs a, cudaStream_t stream) {
  const int slices = (a.d + kCols - 1) / kCols;
  if (slices > 65535) return cudaErrorInvalidValue;
  // Two CTAs for each SM, and no more rows a CTA than it has room for.
  a.classes = std::max({1, 2 * 152 / slices, (a.V + kMaxLocal - 1) / kMaxLocal});
  a.classes = std::min(a.classes, a.V);
  a.inverse = (1ULL << 40) / a.classes + 1;
  a.local = (a.V + a.classes - 1) / a.classes;
  a.chunk = std::min(kChunk, a.T / 32 * 32 + 32);
  const size_t smem = sizeof(GradSmem) + (static_cast<size_t>(a.local) + 1 + 2 * a.chunk) * 4;
  auto kernel = embed_backward_kernel<T, N>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(a.classes, slices), dim3(kGradThreads), smem, stream, a);
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
  GradArgs a{tokens, dout, dtable, T, V, d, 0, 0, scale, accumulate, 0, 0};
  const bool vec = d % 4 == 0 && on16(dtable) && reinterpret_cast<uintptr_t>(dout) % (dout_bf16 ? 8 : 16) == 0;
  if (dout_bf16)
    return vec ? backward_typed<__nv_bfloat16, 4>(a, stream) : backward_typed<__nv_bfloat16, 1>(a, stream);
  return vec ? backward_typed<float, 4>(a, stream) : backward_typed<float, 1>(a, stream);
}

}  // namespace txl
