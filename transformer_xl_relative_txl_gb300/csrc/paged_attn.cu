// The paged attention's dispatch, its tensor maps, and the division of its
// work as the host sees it (a test hook).
#include <algorithm>
#include <cmath>
#include <vector>

#include "paged_tiles.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

template <typename Units>
int pieces_of(int H, int n, const int* start, const int* rows, const int* fresh, int most, int* out, int cap) {
  std::vector<PlanSeq> list(n);
  long long total = 0;
  for (int i = 0; i < n; ++i) {
    list[i] = PlanSeq{total, 0, 0, fresh[i], i, start[i], rows[i]};
    if (fresh[i] > 0) list[i].per = Units::cost_of_head(list[i]);
    total += list[i].per * H;
  }
  const PlanLine line = plan_line(total, plan_ctas<typename Units::Cost>(total, most));
  int count = 0;
  for (int c = 0, x = 0; c < line.ctas; ++c) {
    while (x + 1 < n && list[x + 1].pre <= plan_cut(c, line)) ++x;
    const long long lo = plan_cut(c, line), hi = plan_cut(c + 1, line);
    PlanAt from = Units::place(list[x], lo);
    from.i = x;
    for (bool more = true; more;) {  // 32 at a time, as a warp does
      PlanAt at{};
      for (int r = 0; r < 32 && more; ++r) {
        more = Units::find(list.data(), n, H, from, r, &at);
        if (!more) break;
        const Piece p = Units::piece(list[at.i], at, c, lo, hi, line);
        if (!(more = p.nks > 0)) break;
        if (count == cap) return -1;
        const int row[10] = {c, at.i, at.h, at.qt, p.t0, p.nks, p.first, p.index, p.pieces, plan_place(c, p.index)};
        std::copy(row, row + 10, out + 10 * static_cast<size_t>(count++));
      }
      from = PlanAt{at.i, at.h, at.qt + 1};
    }
  }
  return count;
}

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
  {
    // Four dimensions as the pools', so that one instruction loads boxes of both.
    const cuuint64_t n_r = a.n_r, dims[4] = {D, n_r, H, 1};
    const cuuint64_t strides[3] = {H * D * 2, D * 2, H * D * n_r * 2};
    const cuuint32_t box[4] = {64, 64, 1, 1};
    if (!enc(&m.r, a.r, 4, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const cuuint64_t row[2] = {D * 2, H * D * 2};
  const cuuint64_t tokens[3] = {D, H, static_cast<cuuint64_t>(a.T)};
  const cuuint32_t box_q[3] = {64, 1, kTileQueries}, box_o[3] = {64, 1, 32};
  if (!enc(&m.q, a.q, 3, tokens, row, box_q)) return cudaErrorInvalidValue;
  m.o = m.q;  // stands in where the output is not bf16 and never touched
  if (a.o_bf16 && !enc(&m.o, a.o, 3, tokens, row, box_o)) return cudaErrorInvalidValue;
  // The sign of the scale is the score products' (exact); a zero
  // scale becomes 1e-30, for which every visible exponent rounds to 2^0 in
  // fp32 exactly as with 0, while masked keys keep an exponent of -inf.
  const TileParams p{plan_args(a, wc.status), __builtin_ctz(b.page_rows), a.bias_u, a.bias_v, a.o, a.lse,
                     std::max(std::fabs(a.scale), 1e-30f) * 1.4426950408889634f, a.scale < 0.f,
                     s.tiles.cuts, s.tiles.part, wc.limit_ns, wc.inject_stall};
  return a.D == 64 ? launch_paged_tc64(m, p, a.o_bf16, sms, stream)
                   : launch_paged_tc128(m, p, a.o_bf16, sms, stream);
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

int paged_pieces(int kind, int D, int H, int n, const int* start, const int* rows, const int* fresh, int ctas, int* out,
                 int cap) {
  if (kind == 2) return pieces_of<SimtUnits>(H, n, start, rows, fresh, ctas, out, cap);
  if (kind == 1) return pieces_of<TileUnits>(H, n, start, rows, fresh, ctas, out, cap);
  return D == 64 ? pieces_of<DecodeUnits64>(H, n, start, rows, fresh, ctas, out, cap)
                 : pieces_of<DecodeUnits32>(H, n, start, rows, fresh, ctas, out, cap);
}

size_t paged_workspace_bytes(int n, int T, int H, int D, bool bf16) {
  (void)n, (void)H;
  return plan_space(nullptr, T, D, bf16, nullptr);
}

// fp32: the CUDA cores.  bf16: sequences of up to 4 new tokens by the decode
// kernel, then the others by tiles of 128 queries; then the joins.  Each waits
// for the one ahead.  (max_new is the host's bound: the lengths themselves are
// on the device, and either kernel finds its own.  The decode kernel behind the
// tiles makes a batch without short sequences 2.5 to 3.7 us longer.)
cudaError_t launch_paged_attn(const PagedAttn& a, const WaitCtl& wc, cudaStream_t stream) {
  PlanSpace s;
  plan_space(a.workspace, a.T, a.D, a.bf16, &s);
  const int sms = paged_sms();
  const JoinPart none{nullptr, nullptr, 0, 0};
  cudaError_t e = cudaSuccess;
  if (!a.bf16) {
    e = launch_paged_simt(a, s, sms, wc.status, stream);
    if (e != cudaSuccess) return e;
    return launch_paged_join(a, JoinPart{s.simt.cuts, s.simt.part, kSimtPerSm * sms, kSimtQueries}, none, stream);
  }
  const bool tiles = a.max_new > kDecodeRows;
  e = launch_paged_decode(a, s, sms, tiles, wc, stream);
  if (e == cudaSuccess && tiles) e = launch_tiles(a, s, sms, wc, stream);
  if (e != cudaSuccess) return e;
  return launch_paged_join(a, JoinPart{s.decode.cuts, s.decode.part, kDecodePerSm * sms, kDecodeRows},
                           tiles ? JoinPart{s.tiles.cuts, s.tiles.part, sms, kTileQueries} : none, stream);
}

}  // namespace txl
