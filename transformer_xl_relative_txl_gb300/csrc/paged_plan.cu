// The division of the bf16 paged attention's work (paged_plan.cuh), made on
// the device at the head of each call, and the call's dispatch.
#include <algorithm>
#include <cmath>
#include <vector>

#include "paged_tiles.cuh"
#include "pdl.cuh"

namespace txl {
namespace {

constexpr int kThreads = 1024;

// Inclusive sums of (cost, count) over the CTA; the CTA's sums in totals.
struct Sum {
  long long cost;
  int count;
};
__device__ Sum scan(Sum x, Sum* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x.cost, d);
    const int z = __shfl_up_sync(0xffffffffu, x.count, d);
    if (lane >= d) x.cost += y, x.count += z;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Sum s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s.cost, d);
      const int z = __shfl_up_sync(0xffffffffu, s.count, d);
      if (lane >= d) s.cost += y, s.count += z;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) x.cost += warp_sums[warp - 1].cost, x.count += warp_sums[warp - 1].count;
  return x;
}

template <typename Walk>
__host__ __device__ __forceinline__ long long head_cost(const PlanSeq& s) {
  Walk w;
  w.s = s;
  return w.cost_of_head();
}

// CTA k makes kind k's list: the valid sequences of its kind with the cost of
// those before each, the sequence each CTA of the kernel starts in, zeroed
// counters.
__global__ void __launch_bounds__(kThreads) plan_kernel(const PagedAttn a, const PlanSpace sp, int decode_ctas,
                                                        int tile_ctas, unsigned int* status) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ Sum warp_sums[32];
  __shared__ long long prefix[kThreads];  // costs before the first sequences of the list
  const int kind = blockIdx.x;
  const PageBook& b = a.book;
  PlanSeq* list = sp.seqs[kind];
  Sum before{0, 0};
  for (int i0 = 0; i0 < a.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    PlanSeq s{};
    Sum mine{0, 0};
    if (i < a.n) {
      s.tok0 = a.cu[i];
      s.n = a.cu[i + 1] - s.tok0;
      s.slot = a.slots[i];
      bool ok = s.slot >= 0 && s.slot < b.n_slots && s.n >= 0 && s.n <= a.max_new && s.tok0 >= 0 &&
                static_cast<long long>(s.tok0) + s.n <= a.T;
      if (ok) {
        s.start = b.start[s.slot];
        s.rows = b.rows[s.slot];
        ok = s.start >= 0 && s.start < b.page_rows && s.rows >= 0 && s.rows <= a.n_r &&
             static_cast<long long>(s.start) + s.rows <= static_cast<long long>(b.max_pages) * b.page_rows;
      }
      if (!ok && kind == 0) atomicOr(status, kStatusPagesBit);
      if (ok && s.n > 0 && (s.n <= kDecodeRows) == (kind == 0)) {
        mine.count = 1;
        const long long per = kind != 0 ? head_cost<TileWalk>(s)
                                        : (a.D == 64 ? head_cost<DecodeWalk64>(s) : head_cost<DecodeWalk32>(s));
        mine.cost = per * a.H;
      }
    }
    const Sum upto = scan(mine, warp_sums);
    if (mine.count != 0) {
      s.pre = before.cost + upto.cost - mine.cost;
      const int at = before.count + upto.count - 1;
      list[at] = s;
      if (at < kThreads) prefix[at] = s.pre;
    }
    before.cost += warp_sums[31].cost;
    before.count += warp_sums[31].count;
  }
  const int ctas = kind == 0 ? plan_ctas<DecodeCost>(before.cost, before.count, decode_ctas)
                             : plan_ctas<TileCost>(before.cost, before.count, tile_ctas);
  __syncthreads();
  if (threadIdx.x == 0) sp.heads[kind] = PlanHead{before.cost, before.count, ctas};
  for (int c = threadIdx.x; c < ctas; c += kThreads) {
    const long long lo = c * before.cost / ctas;
    int x = 0, y = before.count - 1;  // the last sequence with pre <= lo
    while (x < y) {
      const int mid = (x + y + 1) >> 1;
      if ((mid < kThreads ? prefix[mid] : list[mid].pre) <= lo)
        x = mid;
      else
        y = mid - 1;
    }
    sp.starts[kind][c] = x;
  }
  if (kind == 0)
    for (int e = threadIdx.x; e < ctas * 4; e += kThreads) sp.counters[e] = 0;
  else
    for (int c = threadIdx.x; c < tile_ctas; c += kThreads) sp.cuts[c].pieces = 0;
}

}  // namespace

int paged_sms() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = __atomic_load_n(&cached[dev], __ATOMIC_RELAXED);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    n = std::min(n, kMaxSms);
    __atomic_store_n(&cached[dev], n, __ATOMIC_RELAXED);
  }
  return n;
}

cudaError_t launch_paged_plan(const PagedAttn& a, const PlanSpace& s, int sms, unsigned int* status,
                              cudaStream_t stream) {
  return launch_dependent(plan_kernel, dim3(a.max_new > kDecodeRows ? 2 : 1), dim3(kThreads), 0, stream, a, s,
                          kDecodePerSm * sms, sms, status);
}

namespace {

template <typename Walk>
int pieces_of(int kind, int H, int n, const int* start, const int* rows, const int* fresh, int most, int* out,
              int cap) {
  std::vector<PlanSeq> list(n);
  PlanHead head{0, n, 0};
  for (int i = 0; i < n; ++i) {
    list[i] = PlanSeq{head.total, 0, fresh[i], i, start[i], rows[i], 0};
    head.total += head_cost<Walk>(list[i]) * H;
  }
  head.ctas = kind == 0 ? plan_ctas<DecodeCost>(head.total, n, most) : plan_ctas<TileCost>(head.total, n, most);
  std::vector<int> starts(std::max(head.ctas, 1));
  for (int c = 0, x = 0; c < head.ctas; ++c) {
    const long long lo = c * head.total / head.ctas;
    while (x + 1 < n && list[x + 1].pre <= lo) ++x;
    starts[c] = x;
  }
  int count = 0;
  for (int c = 0; c < most; ++c) {
    Walk w;
    for (bool more = w.begin(list.data(), head, starts.data(), H, c); more; more = w.next()) {
      if (count == cap) return -1;
      const int row[10] = {c,       w.s.slot,  w.h,       w.qt,       w.p.t0,
                           w.p.nks, w.p.first, w.p.index, w.p.pieces, plan_place(c, w.p.index)};
      std::copy(row, row + 10, out + 10 * static_cast<size_t>(count++));
    }
  }
  return count;
}

}  // namespace

int paged_pieces(int kind, int D, int H, int n, const int* start, const int* rows, const int* fresh, int ctas, int* out,
                 int cap) {
  if (kind != 0) return pieces_of<TileWalk>(kind, H, n, start, rows, fresh, ctas, out, cap);
  return D == 64 ? pieces_of<DecodeWalk64>(kind, H, n, start, rows, fresh, ctas, out, cap)
                 : pieces_of<DecodeWalk32>(kind, H, n, start, rows, fresh, ctas, out, cap);
}

size_t paged_workspace_bytes(int n, int T, int H, int D, bool bf16) {
  (void)H;
  return bf16 ? plan_space(nullptr, n, T, D, nullptr) : 256;
}

namespace {

cudaError_t launch_tiles(const PagedAttn& a, const PlanSpace& s, int sms, const WaitCtl& wc, cudaStream_t stream) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = api_tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const PageBook& b = a.book;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  auto enc = [&](CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t D = a.D, H = a.H, P = b.page_rows;
  TileMaps m;
  {
    const cuuint64_t dims[4] = {D, P, H, static_cast<cuuint64_t>(b.n_pages)};
    const cuuint64_t strides[3] = {D * 2, P * D * 2, H * P * D * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(std::min<cuuint64_t>(P, 64)), 1, 1};
    if (!enc(&m.k, a.kp, 4, dims, strides, box) || !enc(&m.v, a.vp, 4, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  const cuuint64_t row[2] = {D * 2, H * D * 2};
  const cuuint64_t tokens[3] = {D, H, static_cast<cuuint64_t>(a.T)};
  const cuuint32_t box_q[3] = {64, 1, kTileQueries}, box_o[3] = {64, 1, 32};
  if (!enc(&m.q, a.q, 3, tokens, row, box_q)) return cudaErrorInvalidValue;
  {
    // Four dimensions as the pools', so that one instruction loads boxes of both.
    const cuuint64_t n_r = a.n_r, dims[4] = {D, n_r, H, 1};
    const cuuint64_t strides[3] = {H * D * 2, D * 2, H * D * n_r * 2};
    const cuuint32_t box[4] = {64, 64, 1, 1};
    if (!enc(&m.r, a.r, 4, dims, strides, box)) return cudaErrorInvalidValue;
  }
  m.o = m.q;  // stands in where the output is not bf16 and never touched
  if (a.o_bf16 && !enc(&m.o, a.o, 3, tokens, row, box_o)) return cudaErrorInvalidValue;
  // The sign of the scale is folded into (q+u), (q+v) (exact in bf16); a zero
  // scale becomes 1e-30, for which every visible exponent rounds to 2^0 in
  // fp32 exactly as with 0, while masked keys keep an exponent of -inf.
  const TileParams p{b, __builtin_ctz(b.page_rows), a.bias_u, a.bias_v, a.o, a.lse, a.T, a.H,
                     std::max(std::fabs(a.scale), 1e-30f) * 1.4426950408889634f, a.scale < 0.f ? -1.f : 1.f,
                     s.heads + 1, s.seqs[1], s.starts[1], s.cuts, s.part[1], wc.status, wc.limit_ns};
  return a.D == 64 ? launch_paged_tc64(m, p, a.o_bf16, sms, stream)
                   : launch_paged_tc128(m, p, a.o_bf16, sms, stream);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttn& a, const WaitCtl& wc, cudaStream_t stream) {
  if (!a.bf16) return launch_paged_simt(a, wc.status, stream);
  PlanSpace s;
  plan_space(a.workspace, a.n, a.T, a.D, &s);
  const int sms = paged_sms();
  const bool tiles = a.max_new > kDecodeRows;
  cudaError_t e = launch_paged_plan(a, s, sms, wc.status, stream);
  if (e == cudaSuccess && tiles) e = launch_tiles(a, s, sms, wc, stream);
  if (e == cudaSuccess) e = launch_paged_decode(a, s, sms, tiles, wc, stream);
  if (e == cudaSuccess && tiles) e = launch_paged_join(a, s, sms, stream);
  return e;
}

}  // namespace txl
