// bf16 relative attention of new tokens over a paged memory on the tensor
// cores, head dimension 128: tiles of 128 queries of a ragged batch.
//
//   s[t,j] = scale * ((q_t + u) . k_j + (q_t + v) . r_{m+t-j}),  j <= m + t
//   o_t = softmax(s[t,.]) V
//
// The pipeline is that of relattn_tc.cu: three MMA issuers (content score,
// distance score into a three-slot ring of 64-distance tiles, P.V), eight
// softmax warps of which two share a lane quadrant and halve each 64-key step,
// the distance window shifted per lane.  Keys are counted in page rows, the
// work is divided on the device and cut units joined, value rows that are not
// live are zeroed, and only the output is rounded to bf16, as in paged_tc64.cu; the
// weights' second parts lie in shared memory, since tensor memory has no room.
//
// Measured: 8 sequences of 768 tokens over 768 rows, 8 heads, 110 us, 395
// TFLOP/s; 92 us with the roundings of relattn_tc.cu, which leave 3.2e-3 of the
// exact result where this leaves 1.7e-3.  Bound by the step chain of the softmax
// warps, as there.
//
// TMEM (512 columns): O [0,128), P0, P1 [128,192) (bf16 pairs), S0, S1
// [192,320), distance ring [320,512).  Warps: 0-7 softmax (warp w: lane
// quadrant w%4, key columns 32 (w/4) .. + 31); 8 TMA loader; 9 content-score
// MMA issuer (owns the TMEM allocation); 10 PV MMA issuer; 11 distance-score
// MMA issuer.  Every wait is bounded.
#include <cmath>
#include <cstdint>

#include "paged_tiles.cuh"
#include "pdl.cuh"
#include "relattn_tc_common.cuh"
#include "txl_device.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int D = 128;
constexpr int BM = 128;  // query rows per unit (TMEM lanes)
constexpr int BN = 64;   // keys per step, distances per ring tile
constexpr int kLoaderWarp = 8;
constexpr int kMmaWarp = 9;   // S = (q+u)K^T issuer; owns the TMEM allocation
constexpr int kPvWarp = 10;   // O += P V issuer
constexpr int kQrWarp = 11;   // G = (q+v)R^T (distance ring) issuer
constexpr int kThreads = 384;
constexpr uint32_t kColO = 0;
constexpr uint32_t kColP = 128;  // P0, P1: 32 columns each
constexpr uint32_t kColS = 192;  // S0, S1: 64 columns each
constexpr uint32_t kColG = 320;  // distance ring: 3 slots of 64 columns
constexpr int kSlots = 3;
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.0f;  // log2 headroom before the running max moves

constexpr int kChunks = D / 64;
constexpr int kRowChunk = BN * 128;  // 64 rows x 128 B
constexpr int kRowTile = kChunks * kRowChunk;
constexpr int kQChunk = BM * 128;    // 128 rows x 128 B
constexpr int kQTile = kChunks * kQChunk;
constexpr int NK = 2, NV = 2, NR = 2;  // the loader takes one stage count
constexpr int kPTile = BM * 128;        // 128 rows of 64 weights
constexpr int kOffQ = 0;                       // q: 2 buffers
constexpr int kOffK = kOffQ + 2 * kQTile;
constexpr int kOffV = kOffK + NK * kRowTile;
constexpr int kOffR = kOffV + NV * kRowTile;
constexpr int kOffPlo = kOffR + NR * kRowTile;  // P's lo parts (bf16): 2 buffers
constexpr int kOffTermK = kOffPlo + 2 * kPTile;    // bias terms of the K tiles, then of the R tiles
constexpr int kOffTermR = kOffTermK + BiasTerm<D, NK>::kBytes;
constexpr int kOffRed = kOffTermR + BiasTerm<D, NR>::kBytes;
constexpr int kRedFloats = 2 * 2 * BM + 2 * BM;  // [step parity][half][row] maxima, [unit parity][row] sums
constexpr int kOffBar = kOffRed + kRedFloats * 4;
constexpr int kBarBytes = 5120;
constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Bars {
  uint64_t fullK[NK], emptyK[NK], fullV[NV], emptyV[NV], fullR[NR], emptyR[NR];
  uint64_t q_full[2], q_empty[2];  // by unit parity
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], o_full, o_free, g_free[kSlots], mma_final,
      pv_final;
  uint64_t g_full[2], qr_final;  // distance tile of a step ready (per S buffer parity); QR issuer done
  uint64_t xbar[4];  // row-max exchange of warps quad and quad+4 (64 arrivals per step)
  uint64_t lbar[4];  // row-sum hand-over at the end of a unit (32 arrivals)
  TileUnit units[kUnitRing];
  PlanState plan;
  int any;  // the CTA has a unit
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block too large");

template <bool O_BF16, bool STALL>
__global__ void __launch_bounds__(kThreads, 1) paged_tc128_kernel(const __grid_constant__ TileMaps tm, const TileParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  uint8_t* sQ = smem + kOffQ;
  uint8_t* sTermK = smem + kOffTermK;
  uint8_t* sTermR = smem + kOffTermR;
  uint8_t* sK = smem + kOffK;
  uint8_t* sV = smem + kOffV;
  uint8_t* sR = smem + kOffR;
  uint8_t* sPlo = smem + kOffPlo;
  float* red = reinterpret_cast<float*>(smem + kOffRed);
  float* lred = red + 2 * 2 * BM;
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int* abort = &bars->abort;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->fullK[s], 1);
      mbar_init(&bars->emptyK[s], 1);
      mbar_init(&bars->fullV[s], 1);
      mbar_init(&bars->emptyV[s], 1);
      mbar_init(&bars->fullR[s], 1);
      mbar_init(&bars->emptyR[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      if (s < kSlots) mbar_init(&bars->g_free[s], 8);
      mbar_init(&bars->xbar[s], 64);
      mbar_init(&bars->lbar[s], 32);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->g_full[s], 1);
      mbar_init(&bars->s_free[s], 8);
      mbar_init(&bars->p_full[s], 8);
      mbar_init(&bars->pv_done[s], 1);
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 10);  // the softmax warps have seen the unit, both score products are done
    }
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->o_free, 4);
    mbar_init(&bars->mma_final, 1);
    mbar_init(&bars->qr_final, 1);
    mbar_init(&bars->pv_final, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  // What ran before the decode kernel ahead wrote the book, the queries and the
  // pages: its writes, too, are this grid's to see only behind a wait of its own.
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) p.cuts[blockIdx.x] = PlanCut{0, 0, 0, 0};
  plan_begin<TileUnits>(p.args, static_cast<int>(gridDim.x), &bars->plan);
  if (warp != kLoaderWarp) {  // the loader has this barrier behind the first units
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = bars->tmem_base;
  const bool any = bars->any != 0;
  const uint64_t wait_ns = p.wait_ns;

  if (warp == kLoaderWarp) {
    // ============================ TMA loader ===============================
    run_tile_loader<D, NK, true, STALL>(bars, tm, p, sQ, sK, sV, sR);
  } else if (warp == kMmaWarp) {
    // ============================ MMA issuer ===============================
    const uint32_t idS = idesc_bf16(128, BN, false, false) | (p.negative ? kNegateA : 0u);
    // Descriptor bases; the start-address field holds address / 16 in its
    // low 14 bits, so byte offsets inside shared memory are added as
    // offset / 16 (no carry: shared addresses stay below 256 KB).
    const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
    BiasTerm<D, NK> term(sTermK);
    const uint64_t dTerm = term.term_desc(), dOnes = term.ones_desc();
    const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024);
    constexpr uint32_t kTile16 = kRowTile >> 4;
    uint32_t gt = 0, un = 0;  // gt: steps, and K tiles, so far
    bool ok = true;
    while (any && ok) {
      if (!(ok = warp_wait(&bars->q_full[un & 1], (un >> 1) & 1, wait_ns, abort))) break;
      const int nks = bars->units[un % kUnitRing].nks, next_h = bars->units[un % kUnitRing].next_h;
      const uint32_t g0 = gt;
      const uint64_t dq = dQ + (un & 1) * (kQTile >> 4);
      term.load(p.bias_u, bars->units[un % kUnitRing].h);
      for (int t = 0; t < nks; ++t) {
        const uint32_t g = g0 + t, sb = g & 1;
        const int sk = g % NK;
        if (!(ok = warp_wait(&bars->fullK[sk], (g / NK) & 1, wait_ns, abort))) break;
        term.append(sK + sk * kRowTile, sk);
        // S buffer sb was last read by step g-2.
        if (g >= 2 && !(ok = warp_wait(&bars->s_free[sb], ((g - 2) >> 1) & 1, wait_ns, abort))) break;
        if (lane == 0) {
          tc_fence_after();
          mma_scores<D>(tmem + kColS + sb * BN, dq, dK + sk * kTile16, dOnes, dTerm + sk * (kBiasStage >> 4), idS);
          tc_commit(&bars->emptyK[sk]);
          tc_commit(&bars->s_full[sb]);
          if (t == nks - 1) tc_commit(&bars->q_empty[un & 1]);
        }
        __syncwarp();
      }
      if (!ok || next_h < 0) break;
      gt = g0 + nks;
      ++un;
    }
    if (lane == 0) {
      if (!ok) report_timeout(abort, p.args.status);
      tc_commit(&bars->mma_final);
      mbar_wait_own(&bars->mma_final, 0, wait_ns);
    }
  } else if (warp == kPvWarp) {
    // ============================ PV issuer ================================
    constexpr uint32_t idO = idesc_bf16(128, D, false, true);
    const uint64_t dV = sdesc_sw128(smem_u32(sV), kRowChunk, 1024);
    const uint64_t dP = sdesc_sw128(smem_u32(sPlo), 16, 1024);
    constexpr uint32_t kTile16 = kRowTile >> 4;
    uint32_t g = 0, un = 0;  // g: steps, and V tiles, so far
    bool ok = true;
    while (any && ok) {
      // The unit is read behind the barrier of its first V tile.
      int nks = 1, t0 = 0, start = 0, last = 0, next_h = -1;
      for (int t = 0; t < nks; ++t, ++g) {
        const int sv = g % NV;
        if (!(ok = warp_wait(&bars->fullV[sv], (g / NV) & 1, wait_ns, abort))) break;
        if (t == 0) {
          const TileUnit& w = bars->units[un % kUnitRing];
          nks = w.nks;
          t0 = w.t0;
          start = w.start;
          last = w.last;
          next_h = w.next_h;
          if (STALL && blockIdx.x % 2 != 0) nks = 1, next_h = -1;
        }
        zero_dead_rows<D>(start, last, t0 + t, sV + sv * kRowTile, lane);
        if (!(ok = warp_wait(&bars->p_full[g & 1], (g >> 1) & 1, wait_ns, abort))) break;
        if (t == 0 && un > 0 && !(ok = warp_wait(&bars->o_free, (un - 1) & 1, wait_ns, abort))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dv = dV + sv * kTile16;
          const uint32_t pa = tmem + kColP + (g & 1) * 32;
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + kColO, pa + kk * 8, dv + ((kk * 16 * 128) >> 4), idO, (t > 0 || kk > 0) ? 1u : 0u);
          const uint64_t dp = dP + (g & 1) * (kPTile >> 4);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) mma_ss(tmem + kColO, dp + kk * 2, dv + ((kk * 16 * 128) >> 4), idO, 1);
          tc_commit(&bars->emptyV[sv]);
          tc_commit(&bars->pv_done[g & 1]);
          if (t == nks - 1) tc_commit(&bars->o_full);
        }
        __syncwarp();
      }
      if (!ok || next_h < 0) break;
      ++un;
    }
    if (lane == 0) {
      if (any && !ok) report_timeout(abort, p.args.status);
      tc_commit(&bars->pv_final);
      mbar_wait_own(&bars->pv_final, 0, wait_ns);
    }
  } else if (warp == kQrWarp) {
    // ========================= distance-ring issuer =========================
    // G tile e = (q+v) R_e^T into ring slot (e+2) % 3 once the softmax has
    // released the slot's previous tile; tiles -2 and -1 of a unit with its
    // first step.  Its own thread, so the ring never waits behind the S
    // MMAs' barriers (and the reverse); it commits g_full per step.
    const uint32_t idS = idesc_bf16(128, BN, false, false) | (p.negative ? kNegateA : 0u);
    const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
    BiasTerm<D, NR> term(sTermR);
    const uint64_t dTerm = term.term_desc(), dOnes = term.ones_desc();
    const uint64_t dR = sdesc_sw128(smem_u32(sR), 16, 1024);
    constexpr uint32_t kTile16 = kRowTile >> 4;
    uint32_t nR = 0, gt = 0, un = 0;
    uint32_t gsu0 = 0, gsu1 = 0, gsu2 = 0;  // writes per ring slot so far
    bool ok = true;
    while (any && ok) {
      if (!(ok = warp_wait(&bars->q_full[un & 1], (un >> 1) & 1, wait_ns, abort))) break;
      const int nks = bars->units[un % kUnitRing].nks, next_h = bars->units[un % kUnitRing].next_h;
      const uint32_t g0 = gt;
      const uint64_t dq = dQ + (un & 1) * (kQTile >> 4);
      term.load(p.bias_v, bars->units[un % kUnitRing].h);
      for (int t = 0; t < nks; ++t) {
        const uint32_t g = g0 + t, sb = g & 1;
        for (int e = (t == 0 ? -2 : t); e <= t; ++e) {
          const int sr = nR % NR;
          if (!(ok = warp_wait(&bars->fullR[sr], (nR / NR) & 1, wait_ns, abort))) break;
          term.append(sR + sr * kRowTile, sr);
          const int slot = (e + 2) % kSlots;
          const uint32_t used = slot == 0 ? gsu0 : (slot == 1 ? gsu1 : gsu2);
          if (used > 0 && !(ok = warp_wait(&bars->g_free[slot], (used - 1) & 1, wait_ns, abort))) break;
          if (lane == 0) {
            tc_fence_after();
            mma_scores<D>(tmem + kColG + slot * BN, dq, dR + sr * kTile16, dOnes, dTerm + sr * (kBiasStage >> 4), idS);
            tc_commit(&bars->emptyR[sr]);
          }
          ++nR;
          gsu0 += slot == 0;
          gsu1 += slot == 1;
          gsu2 += slot == 2;
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) {
          tc_commit(&bars->g_full[sb]);
          if (t == nks - 1) tc_commit(&bars->q_empty[un & 1]);
        }
        __syncwarp();
      }
      if (!ok || next_h < 0) break;
      gt = g0 + nks;
      ++un;
    }
    if (lane == 0) {
      if (!ok) report_timeout(abort, p.args.status);
      tc_commit(&bars->qr_final);
      mbar_wait_own(&bars->qr_final, 0, wait_ns);
    }
  } else {
    // ============================ softmax warps ============================
    const int half = warp >> 2;  // 0: key columns 0-31 of a step, 1: columns 32-63
    const int quad = warp & 3;   // TMEM lane quadrant
    const int a = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const float sl2 = p.scale_log2e;
    uint32_t gt = 0, un = 0;
    bool ok = true;

    while (any && ok) {
      // Published before the q tile was loaded.
      if (!(ok = warp_wait(&bars->q_full[un & 1], (un >> 1) & 1, wait_ns, abort))) break;
      const TileUnit* unit = &bars->units[un % kUnitRing];
      const int nks = unit->nks, t0 = unit->t0, d0 = unit->d0, start = unit->start;
      const bool has_next = unit->next_h >= 0;
      warp_arrive(&bars->q_empty[un & 1]);
      float m_use = -INFINITY;  // running max in log2 units (lazy)
      float l_half = 0.f;       // row sum over this half's columns
      const uint32_t g0 = gt;
      for (int t = 0; t < nks; ++t) {
        const uint32_t g = g0 + t, sb = g & 1;
        if (!(ok = warp_wait(&bars->s_full[sb], (g >> 1) & 1, wait_ns, abort))) break;
        if (!(ok = warp_wait(&bars->g_full[sb], (g >> 1) & 1, wait_ns, abort))) break;
        tc_fence_after();
        uint32_t sraw[32], x0[32], x1[32];
        tmem_ld32(tmem + lane_base + kColS + sb * BN + 32 * half, sraw);
        // Distance window of this warp: ring-relative index z = 64 + a - c
        // (z < 64: tile t, < 128: tile t-1, else tile t-2); the warp reads
        // z in [zq, zq + 64) and lane l uses z = zq + 32 + l - k for column k.
        const int zq = 32 * (1 + quad - half);
        const uint32_t c0 = kColG + ((t - (zq >> 6) + 2) % kSlots) * BN + (zq & 63);
        const uint32_t c1 = kColG + ((t - ((zq + 32) >> 6) + 2) % kSlots) * BN + ((zq + 32) & 63);
        tmem_ld32(tmem + lane_base + c0, x0);
        tmem_ld32(tmem + lane_base + c1, x1);
        tmem_wait_ld(sraw);
        tmem_wait_ld(x0);
        tmem_wait_ld(x1);
        warp_arrive_tc(&bars->s_free[sb]);              // S buffer may be refilled
        warp_arrive_tc(&bars->g_free[t % kSlots]);      // distance tile t-2: last read
        // x[k] = content + distance score of key column 32*half + k
        float x[32];
        {
          uint32_t bd[32];
          window_shift_f32(x0, x1, lane, bd);
          add_columns(sraw, bd, x);
        }
        const int kt = t0 + t;                           // key step of the tile
        const int lim = d0 - BN * kt + a - 32 * half;    // column k visible iff low <= k <= lim
        const int low = start - BN * kt - 32 * half;
        if (low > 0 || d0 - BN * kt + quad * 32 - 32 * half < 31) {  // some lane of the warp masks
          const uint32_t v = visible_columns(low, lim);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = v >> k & 1 ? x[k] : -INFINITY;
        }
        float t3[11];
#pragma unroll
        for (int n = 0; n < 10; ++n) t3[n] = max3f(x[3 * n], x[3 * n + 1], x[3 * n + 2]);
        t3[10] = fmaxf(x[30], x[31]);
        float mx = max3f(max3f(t3[0], t3[1], t3[2]), max3f(t3[3], t3[4], t3[5]),
                         max3f(max3f(t3[6], t3[7], t3[8]), t3[9], t3[10]));
        // row max over both halves of the step
        float* rs = red + (g & 1) * 2 * BM;
        rs[half * BM + a] = mx;
        mbar_arrive(&bars->xbar[quad]);
        if (!(ok = warp_wait(&bars->xbar[quad], g & 1, wait_ns, abort))) break;
        mx = fmaxf(mx, rs[(1 - half) * BM + a]) * sl2;
        float m_new = m_use, alpha = 1.f;
        if (mx > m_use + kLazy) {
          m_new = mx;
          alpha = ex2(m_use - mx);
        }
        // A row with no visible key yet keeps m_new = -inf; its exponents are
        // then taken against 0 (all -inf, so every p is 0).
        const float m_eff = m_new == -INFINITY ? 0.f : m_new;
        uint32_t pk[16], pl[16];
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-m_eff, -m_eff);
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float2 y = __ffma2_rn(make_float2(x[2 * n], x[2 * n + 1]), sc2, nm2);
          const float2 e = make_float2(ex2(y.x), ex2(y.y));
          if (n & 1)
            acc1 = __fadd2_rn(acc1, e);
          else
            acc0 = __fadd2_rn(acc0, e);
          split_weights(e, pk[n], pl[n]);
        }
        l_half = l_half * alpha + ((acc0.x + acc0.y) + (acc1.x + acc1.y));
        if (half == 0 && t > 0 && __any_sync(0xffffffffu, alpha < 1.f)) {
          // O holds PV up to step t-1; rescale once that PV has completed.
          if (!(ok = warp_wait(&bars->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, wait_ns, abort))) break;
          tc_fence_after();
#pragma unroll
          for (int oc = 0; oc < D / 32; ++oc) {
            uint32_t ov[32];
            tmem_ld32(tmem + lane_base + kColO + oc * 32, ov);
            tmem_wait_ld(ov);
#pragma unroll
            for (int n = 0; n < 32; ++n) ov[n] = __float_as_uint(__uint_as_float(ov[n]) * alpha);
            tmem_st32(tmem + lane_base + kColO + oc * 32, ov);
          }
        }
        m_use = m_new;
        // P buffer sb was last read by the PV of step g-2.
        if (g >= 2 && !(ok = warp_wait(&bars->pv_done[sb], ((g - 2) >> 1) & 1, wait_ns, abort))) break;
        tc_fence_after();
        tmem_st16(tmem + lane_base + kColP + sb * 32 + 16 * half, pk);
        uint8_t* prow = sPlo + sb * kPTile + (a / 8) * 1024 + (a % 8) * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(prow + (((4 * half + c) ^ (a % 8)) * 16)) =
              make_uint4(pl[4 * c], pl[4 * c + 1], pl[4 * c + 2], pl[4 * c + 3]);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive_smem(&bars->p_full[sb]);
      }
      if (!ok) break;
      // Distance tiles nks-2 and nks-1 are not read any more in this unit.
      warp_arrive_tc(&bars->g_free[nks % kSlots]);
      warp_arrive_tc(&bars->g_free[(nks + 1) % kSlots]);
      float* ls = lred + (un & 1) * BM;
      if (half == 1) {
        ls[a] = l_half;
        mbar_arrive(&bars->lbar[quad]);
      }
      if (half == 0) {
        if (!(ok = warp_wait(&bars->lbar[quad], un & 1, wait_ns, abort))) break;
        const float l = l_half + ls[a];
        if (!(ok = warp_wait(&bars->o_full, un & 1, wait_ns, abort))) break;
        tc_fence_after();
        const bool seen = m_use != -INFINITY;  // the row sees a key of this piece
        const float inv_l = seen ? 1.f / l : 0.f;
        const float lse2 = seen ? m_use + __log2f(l) : -INFINITY;
        const TileUnit w = *unit;
        store_lse(w, a, lse2, p.lse, p.part, p.args.T, D);
#pragma unroll 1
        for (int oc = 0; oc < D / 32; ++oc) {
          uint32_t tmp[32];
          float ov[32];
          tmem_ld32(tmem + lane_base + kColO + oc * 32, tmp);
          tmem_wait_ld(tmp);
          if (oc == D / 32 - 1) warp_arrive_tc(&bars->o_free);
#pragma unroll
          for (int n = 0; n < 32; ++n) ov[n] = __uint_as_float(tmp[n]) * inv_l;
          store_columns<D, O_BF16>(w, a, oc, ov, p.o, p.part, p.args.H);
        }
      }
      if (!has_next) break;
      gt = g0 + nks;
      ++un;
    }
    if (!ok) report_timeout(abort, p.args.status);
  }

  // ---- teardown ------------------------------------------------------------
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool O_BF16, bool STALL>
cudaError_t launch(const TileMaps& m, const TileParams& p, int sms, cudaStream_t stream) {
  auto kern = paged_tc128_kernel<O_BF16, STALL>;
  static unsigned configured = 0;  // one bit per device ordinal < 32
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1u << dev))) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)) != cudaSuccess)
      return e;
    if (dev < 32) __atomic_fetch_or(&configured, 1u << dev, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, dim3(sms), dim3(kThreads), kSmemBytes, stream, m, p);
}

}  // namespace

cudaError_t launch_paged_tc128(const TileMaps& m, const TileParams& p, bool o_bf16, int sms, cudaStream_t stream) {
  if (p.inject_stall) return o_bf16 ? launch<true, true>(m, p, sms, stream) : launch<false, true>(m, p, sms, stream);
  return o_bf16 ? launch<true, false>(m, p, sms, stream) : launch<false, false>(m, p, sms, stream);
}

}  // namespace txl
