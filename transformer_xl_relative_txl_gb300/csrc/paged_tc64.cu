// bf16 relative attention of new tokens over a paged memory on the tensor
// cores, head dimension 64: tiles of 128 queries of a ragged batch.
//
//   s[t,j] = scale * ((q_t + u) . k_j + (q_t + v) . r_{m+t-j}),  j <= m + t
//   o_t = softmax(s[t,.]) V
//
// The pipeline is that of relattn_tc64.cu: three MMA issuers (content score,
// distance score into a ring of 64-distance tiles, P.V), eight softmax warps
// that take alternate 64-key steps, the distance window shifted per lane, two
// output accumulators merged at the end of a unit.  What is of its own:
//
//   * Keys are counted in page rows, from the slot's first page, so a 64-row
//     key tile is a box of one page (or 2 or 4 boxes of smaller pages) and
//     never straddles more; rows before the first live one are masked, and
//     distances are differences of page rows.
//   * The division of the work comes from the device (paged_plan.cuh): equal
//     ranges of key steps per CTA, so that ragged lengths, few sequences and
//     long memories are all one case; a unit that a range cuts is joined
//     through the workspace.  The loader publishes the units (paged_tiles.cuh).
//   * Value rows that are not live are zeroed in shared memory by the P.V
//     issuer's warp.
//   * A 32-row box of output whose rows are all the unit's leaves by TMA, the
//     last rows of a sequence by plain stores.
//
// Rounded to bf16: the output alone.  q is an operand as it comes, the bias terms
// are added apart (paged_tiles.cuh), the distance scores pass the shift in fp32,
// the weights are two bf16 parts each (P.V twice); scores, maxima, sums and
// accumulators are fp32.  That is 1.7e-3 of the exact result (relative L2).  With
// (q+u), (q+v), the distance scores and the weights rounded to bf16, as
// relattn_tc64.cu has them, it was 3.2e-3, and 89 us for what now takes 104.
//
// Measured: 22 sequences of 512 tokens over 512 rows, 8 heads, 104 us, 256
// TFLOP/s counted without the distances that the shift leaves out.  Bound by
// the softmax warps, about 1300 instructions a step, which keep the ALU pipe 53%
// busy (the tensor pipe is 24% busy, DRAM 8%).
//
// TMEM (512 columns): O0 [0,64) O1 [64,128) S0 [128,192) S1 [192,256)
// distance ring [256,512).  Warps: 0-7 softmax (warp w: lane quadrant w%4,
// step parity w/4); 8 TMA loader; 9 content-score MMA issuer (owns the TMEM
// allocation); 10 PV MMA issuer; 11 distance-score MMA issuer.  Every wait is
// bounded; a wait that runs out raises a CTA abort flag and the device status
// word, every role unwinds and the TMEM is freed before exit.
#include <cmath>
#include <cstdint>

#include "paged_tiles.cuh"
#include "pdl.cuh"
#include "relattn_tc_common.cuh"
#include "txl_device.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int BM = kTileRows;
constexpr int BN = kStepKeys;
constexpr int D = 64;
constexpr int kLoaderWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kPvWarp = 10;
constexpr int kQrWarp = 11;
constexpr int kThreads = 384;  // 3 warpgroups: 2 softmax, 1 producer (loader, three MMA issuers)
// Register split (launch: 168 per thread, 384 x 168 = 64512): softmax
// warpgroups 192, producer warpgroup 120; 2*128*192 + 128*120 = 64512.  (22
// sequences of 512 tokens over 512 rows, and a mixed batch: 104.4 and 103.0 us;
// 104.3 and 104.7 with 208 and 88, 108.2 and 107.0 with 200 and 104, 109.5 and 110.2
// with 216 and 72.)
constexpr uint32_t kRegsSoftmax = 192;
constexpr uint32_t kRegsProducer = 120;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsProducer <= kThreads * 168, "register split");
constexpr uint32_t kColO = 0;    // O0, O1: 64 columns each
constexpr uint32_t kColS = 128;  // S0, S1: 64 columns each
constexpr uint32_t kColG = 256;  // distance ring: 4 slots of 64 columns
constexpr int kSlots = 4;
static_assert(kSlots == 4, "ring slot counters and barrier init assume four slots");
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.0f;  // log2 headroom before a running max moves

constexpr int kRowTile = BN * 128;  // 64 rows x 64 bf16 (8 KB)
constexpr int kQTile = BM * 128;    // 128 rows x 64 bf16 (16 KB)
constexpr int NK = 4, NV = 4, NR = 4;  // K, V, R tile stages
static_assert(NK == NV && NK == NR, "the loader takes one stage count");
constexpr int kOffQ = 0;                        // q: 2 buffers
constexpr int kOffK = kOffQ + 2 * kQTile;
constexpr int kOffV = kOffK + NK * kRowTile;
constexpr int kOffR = kOffV + NV * kRowTile;
constexpr int kOffP = kOffR + NR * kRowTile;    // P (bf16), hi parts: 2 buffers, same layout as q
constexpr int kOffPlo = kOffP + 2 * kQTile;     // lo parts
constexpr int kOffTermK = kOffPlo + 2 * kQTile;  // bias terms of the K tiles, then of the R tiles
constexpr int kOffTermR = kOffTermK + BiasTerm<D, NK>::kBytes;
constexpr int kOffRed = kOffTermR + BiasTerm<D, NR>::kBytes;  // [unit parity][m, l][row] handed to the epilogue
constexpr int kOffBar = kOffRed + 2 * 2 * BM * 4;
constexpr int kBarBytes = 5120;
constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Bars {
  uint64_t fullK[NK], emptyK[NK], fullV[NV], emptyV[NV], fullR[NR], emptyR[NR];
  uint64_t q_full[2], q_empty[2];  // by unit parity
  uint64_t s_full[2], p_full[2], pv_done[2], o_full, o_free;
  uint64_t sread[4];  // step g's S and distance window have been read (index g % 4, phase g / 4)
  uint64_t mma_final, pv_final, qr_final;
  uint64_t lbar[4];   // per quadrant: the non-owning warp's (m, l) of a unit is in `red`
  uint64_t lfree[4];  // per quadrant: the epilogue has read it
  TileUnit units[kUnitRing];
  PlanState plan;
  int any;            // the CTA has a unit
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block too large");

template <bool O_BF16, bool STALL>
__global__ void __launch_bounds__(kThreads, 1) paged_tc64_kernel(const __grid_constant__ TileMaps tm, const TileParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  uint8_t* sQ = smem + kOffQ;
  uint8_t* sTermK = smem + kOffTermK;
  uint8_t* sTermR = smem + kOffTermR;
  uint8_t* sK = smem + kOffK;
  uint8_t* sV = smem + kOffV;
  uint8_t* sR = smem + kOffR;
  uint8_t* sP = smem + kOffP;
  float* red = reinterpret_cast<float*>(smem + kOffRed);
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int* abort = &bars->abort;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars->fullK[s], 1);
      mbar_init(&bars->emptyK[s], 1);
      mbar_init(&bars->fullV[s], 1);
      mbar_init(&bars->emptyV[s], 1);
      mbar_init(&bars->fullR[s], 1);
      mbar_init(&bars->emptyR[s], 1);
      mbar_init(&bars->lbar[s], 32);
      mbar_init(&bars->lfree[s], 1);
      mbar_init(&bars->sread[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->s_full[s], 2);  // content and distance MMAs of a step
      mbar_init(&bars->p_full[s], 4);
      mbar_init(&bars->pv_done[s], 1);
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 10);  // the softmax warps have seen the unit, both score products are done
    }
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->o_free, 4);
    mbar_init(&bars->mma_final, 1);
    mbar_init(&bars->pv_final, 1);
    mbar_init(&bars->qr_final, 1);
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
    setmaxnreg_dec<kRegsProducer>();
    run_tile_loader<D, NK, false, STALL>(bars, tm, p, sQ, sK, sV, sR);
  } else if (warp == kMmaWarp) {
    // ===================== content-score MMA issuer ========================
    setmaxnreg_dec<kRegsProducer>();
    const uint32_t idS = idesc_bf16(128, BN, false, false) | (p.negative ? kNegateA : 0u);
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
        if (g >= 2 && !(ok = warp_wait(&bars->sread[(g - 2) & 3], ((g - 2) >> 2) & 1, wait_ns, abort))) break;
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
  } else if (warp == kQrWarp) {
    // ==================== distance-score MMA issuer ========================
    setmaxnreg_dec<kRegsProducer>();
    const uint32_t idS = idesc_bf16(128, BN, false, false) | (p.negative ? kNegateA : 0u);
    const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
    BiasTerm<D, NR> term(sTermR);
    const uint64_t dTerm = term.term_desc(), dOnes = term.ones_desc();
    const uint64_t dR = sdesc_sw128(smem_u32(sR), 16, 1024);
    constexpr uint32_t kTile16 = kRowTile >> 4;
    uint32_t nR = 0, gt = 0, un = 0;
    // Last global step that reads the tile now in each ring slot (-1: none).
    int last0 = -1, last1 = -1, last2 = -1, last3 = -1;
    int rb = 0;  // ring slot of the first distance tile (-2) of the unit
    bool ok = true;
    while (any && ok) {
      if (!(ok = warp_wait(&bars->q_full[un & 1], (un >> 1) & 1, wait_ns, abort))) break;
      const int nks = bars->units[un % kUnitRing].nks, next_h = bars->units[un % kUnitRing].next_h;
      const uint32_t g0 = gt;
      const uint64_t dq = dQ + (un & 1) * (kQTile >> 4);
      term.load(p.bias_v, bars->units[un % kUnitRing].h);
      for (int t = 0; ok && t < nks; ++t) {
        const uint32_t sb = (g0 + t) & 1;
        for (int e = (t == 0 ? -2 : t); e <= t; ++e) {
          const int sr = nR % NR;
          if (!(ok = warp_wait(&bars->fullR[sr], (nR / NR) & 1, wait_ns, abort))) break;
          term.append(sR + sr * kRowTile, sr);
          const int slot = (rb + e + 2) & (kSlots - 1);
          // The slot's previous tile is free once every step up to its
          // last reader L has read: steps of one parity read in order, so
          // waiting for steps L and L-1 covers both parities.  (Four
          // barriers by step % 4 keep these waits from aliasing: step L+3
          // cannot have read before this tile exists.)
          const int L = slot == 0 ? last0 : (slot == 1 ? last1 : (slot == 2 ? last2 : last3));
          if (L >= 0 && !(ok = warp_wait(&bars->sread[L & 3], (L >> 2) & 1, wait_ns, abort))) break;
          if (L >= 1 && !(ok = warp_wait(&bars->sread[(L - 1) & 3], ((L - 1) >> 2) & 1, wait_ns, abort))) break;
          if (lane == 0) {
            tc_fence_after();
            mma_scores<D>(tmem + kColG + slot * BN, dq, dR + sr * kTile16, dOnes, dTerm + sr * (kBiasStage >> 4), idS);
            tc_commit(&bars->emptyR[sr]);
          }
          ++nR;
          const int lr = static_cast<int>(g0) + min(e + 2, nks - 1);  // tile e's last reader
          last0 = slot == 0 ? lr : last0;
          last1 = slot == 1 ? lr : last1;
          last2 = slot == 2 ? lr : last2;
          last3 = slot == 3 ? lr : last3;
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) {
          tc_commit(&bars->s_full[sb]);
          if (t == nks - 1) tc_commit(&bars->q_empty[un & 1]);
        }
        __syncwarp();
      }
      if (!ok || next_h < 0) break;
      gt = g0 + nks;
      ++un;
      rb = (rb + nks + 2) & (kSlots - 1);
    }
    if (lane == 0) {
      if (!ok) report_timeout(abort, p.args.status);
      tc_commit(&bars->qr_final);
      mbar_wait_own(&bars->qr_final, 0, wait_ns);
    }
  } else if (warp == kPvWarp) {
    // ============================ PV issuer ================================
    setmaxnreg_dec<kRegsProducer>();
    constexpr uint32_t idO = idesc_bf16(128, D, false, true);
    const uint64_t dV = sdesc_sw128(smem_u32(sV), BN * 128, 1024);
    const uint64_t dP = sdesc_sw128(smem_u32(sP), 16, 1024);
    constexpr uint32_t kLo16 = (kOffPlo - kOffP) >> 4;
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
        // The first PV into each accumulator of a unit overwrites it: the
        // previous unit's epilogue must have read both.
        if (t < 2 && un > 0 && !(ok = warp_wait(&bars->o_free, (un - 1) & 1, wait_ns, abort))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dv = dV + sv * kTile16;
          const uint64_t dp = dP + (g & 1) * (kQTile >> 4);
          const uint32_t od = tmem + kColO + (g & 1) * D;
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ss(od, dp + kk * 2, dv + ((kk * 16 * 128) >> 4), idO, t >= 2 || kk > 0);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) mma_ss(od, dp + kLo16 + kk * 2, dv + ((kk * 16 * 128) >> 4), idO, 1);
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
  } else {
    // ============================ softmax warps ============================
    setmaxnreg_inc<kRegsSoftmax>();
    const int par = warp >> 2;  // step parity taken by this warp
    const int quad = warp & 3;  // TMEM lane quadrant
    const int a = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const float sl2 = p.scale_log2e;
    uint32_t gt = 0, un = 0;
    int rb = 0;  // ring slot of the unit's distance tile -2 (continues across units)
    bool store_pending = false;  // lane 0 has a TMA store out of this warp's P quadrant
    bool ok = true;

    while (any && ok) {
      // Published before the q tile was loaded.
      if (!(ok = warp_wait(&bars->q_full[un & 1], (un >> 1) & 1, wait_ns, abort))) break;
      const TileUnit* unit = &bars->units[un % kUnitRing];
      const int nks = unit->nks, t0 = unit->t0, d0 = unit->d0, start = unit->start;
      const bool has_next = unit->next_h >= 0;
      warp_arrive(&bars->q_empty[un & 1]);
      const uint32_t g0 = gt;
      const int tl = nks - 1;
      const int first = (par - static_cast<int>(g0)) & 1;  // first local step of this warp
      float m_use = -INFINITY;  // running max in log2 units (lazy)
      float l_run = 0.f;
      for (int t = first; t <= tl; t += 2) {
        const uint32_t g = g0 + t, sb = g & 1;
        if (!(ok = warp_wait(&bars->s_full[sb], (g >> 1) & 1, wait_ns, abort))) break;
        tc_fence_after();
        // Distance window of this warp: ring-relative index z = 64 + a - c
        // (z < 64: tile t, < 128: tile t-1, else tile t-2).  Columns 0-31 use
        // z in [32 quad + 32, 32 quad + 96), columns 32-63 z in
        // [32 quad, 32 quad + 64); lane l of column k (within its half) sits
        // at window position l + 32 - k.
        auto zcol = [&](int z) -> uint32_t {
          return kColG + ((rb + t - (z >> 6) + 2) & (kSlots - 1)) * BN + (z & 63);
        };
        const uint32_t sc = tmem + lane_base + kColS + sb * BN;
        const int kt = t0 + t;              // key step of the tile
        const int lim = d0 - BN * kt + a;   // column c visible iff low <= c <= lim
        const int low = start - BN * kt;
        const bool diag = d0 - BN * kt + quad * 32 < 63;  // some lane of the warp masks
        const float m_old = m_use;
        float m_new = m_use;
        // Scores, half of the columns a turn, back into their place in tensor memory;
        // then, the maximum known, the weights, half a turn.  The step's code is what
        // bounds it otherwise: with all 64 columns in a line, in registers, 14% longer
        // for 22 sequences of 512 tokens over 512 rows, a quarter of the warps' waiting
        // for instructions, an eighth so.  (The weights in quarters 5% longer, the scores
        // alone in halves 25%.)
        float mx = -INFINITY;
#pragma unroll 1
        for (int hc = 0; hc < 64; hc += 32) {
          uint32_t s32[32], w0[32], w1[32], bd[32];
          tmem_ld32(tmem + lane_base + zcol(32 * quad + 32 - hc), w0);
          tmem_ld32(tmem + lane_base + zcol(32 * quad + 64 - hc), w1);
          tmem_ld32(sc + hc, s32);
          tmem_wait_ld(w0);
          tmem_wait_ld(w1);
          tmem_wait_ld(s32);
          float x[32];
          window_shift_f32(w0, w1, lane, bd);
          add_columns(s32, bd, x);
          if (diag || low > 0) {
            const uint32_t v = visible_columns(low - hc, lim - hc);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = v >> k & 1 ? x[k] : -INFINITY;
          }
          float t3[11];
#pragma unroll
          for (int n = 0; n < 10; ++n) t3[n] = max3f(x[3 * n], x[3 * n + 1], x[3 * n + 2]);
          t3[10] = fmaxf(x[30], x[31]);
          mx = fmaxf(mx, max3f(max3f(t3[0], t3[1], t3[2]), max3f(t3[3], t3[4], t3[5]),
                               max3f(max3f(t3[6], t3[7], t3[8]), t3[9], t3[10])));
#pragma unroll
          for (int k = 0; k < 32; ++k) s32[k] = __float_as_uint(x[k]);
          tmem_st32(sc + hc, s32);
        }
        tmem_wait_st();
        mx *= sl2;
        if (mx > m_new + kLazy) m_new = mx;
        const float alpha = (m_old == -INFINITY) ? 0.f : ex2(m_old - m_new);  // m_new >= m_old
        // The PV of step g-2 (same P buffer, same accumulator) must be done
        // before P is overwritten or O rescaled.
        if (g >= 2 && !(ok = warp_wait(&bars->pv_done[sb], ((g - 2) >> 1) & 1, wait_ns, abort))) break;
        tc_fence_after();
        if (t > first && __any_sync(0xffffffffu, m_new > m_old)) {
          // O of this parity holds PV up to step t-2; rescale it in place.
          const uint32_t oc0 = tmem + lane_base + kColO + par * D;
#pragma unroll
          for (int oc = 0; oc < D / 32; ++oc) {
            uint32_t ov[32];
            tmem_ld32(oc0 + oc * 32, ov);
            tmem_wait_ld(ov);
#pragma unroll
            for (int n = 0; n < 32; ++n) ov[n] = __float_as_uint(__uint_as_float(ov[n]) * alpha);
            tmem_st32(oc0 + oc * 32, ov);
          }
          tmem_wait_st();
        }
        m_use = m_new;
        if (store_pending) {  // the last epilogue staged its output here
          if (lane == 0) bulk_wait_group_read0();
          __syncwarp();
          store_pending = false;
        }
        // A row with no visible key yet keeps m_new = -inf; its exponents are
        // then taken against 0 (all -inf, so every p is 0).
        const float m_eff = (m_new == -INFINITY) ? 0.f : m_new;
        float sum;
        {
          // Exponentials, their row sum, and the P row a into buffer sb
          // (128B-swizzled K-major, as q), eight columns per store.
          uint8_t* prow = sP + sb * kQTile + (a / 8) * 1024 + (a % 8) * 128;
          float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
          const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-m_eff, -m_eff);
#pragma unroll 1
          for (int hc = 0; hc < 64; hc += 32) {
            uint32_t x[32];
            tmem_ld32(sc + hc, x);
            tmem_wait_ld(x);
            if (hc != 0) warp_arrive_tc(&bars->sread[g & 3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t pk[4], pl[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int n = 4 * c + i;
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[2 * n]), __uint_as_float(x[2 * n + 1])), sc2, nm2);
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                if (i & 1)
                  acc1 = __fadd2_rn(acc1, e);
                else
                  acc0 = __fadd2_rn(acc0, e);
                split_weights(e, pk[i], pl[i]);
              }
              uint8_t* at = prow + (((hc / 8 + c) ^ (a % 8)) * 16);
              *reinterpret_cast<uint4*>(at) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
              *reinterpret_cast<uint4*>(at + (kOffPlo - kOffP)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
            }
          }
          sum = (acc0.x + acc0.y) + (acc1.x + acc1.y);
        }
        l_run = l_run * alpha + sum;
        tc_fence_before();  // orders the O rescale's tcgen05.st before the arrive
        warp_arrive_smem(&bars->p_full[sb]);
      }
      if (!ok) break;
      // The warps of the unit's last step merge the two accumulators and
      // write the output; the other parity hands over its (m, l) and moves on
      // to the next unit, whose first step is its own.
      float* rm = red + (un & 1) * 2 * BM;
      const int owner = static_cast<int>((g0 + tl) & 1);
      if (par != owner) {
        // The owner of the previous unit has read that unit's (m, l).
        if (un > 0 && !(ok = warp_wait(&bars->lfree[quad], (un - 1) & 1, wait_ns, abort))) break;
        rm[a] = m_use;
        rm[BM + a] = l_run;
        mbar_arrive(&bars->lbar[quad]);
      } else {
        if (!(ok = warp_wait(&bars->lbar[quad], un & 1, wait_ns, abort))) break;
        const float m1 = rm[a], l1 = rm[BM + a];
        warp_arrive(&bars->lfree[quad]);
        if (!(ok = warp_wait(&bars->o_full, un & 1, wait_ns, abort))) break;
        tc_fence_after();
        // merge this parity's accumulator (0) with the other's (1)
        const bool has0 = first <= tl;        // this warp had steps
        const bool has1 = (first ^ 1) <= tl;  // the other parity's warp had steps
        const float m = fmaxf(has0 ? m_use : -INFINITY, has1 ? m1 : -INFINITY);
        const bool seen = m != -INFINITY;  // the row sees a key of this piece
        const float a0 = (has0 && seen) ? ex2(m_use - m) : 0.f;
        const float a1 = (has1 && seen) ? ex2(m1 - m) : 0.f;
        const float l = a0 * l_run + a1 * l1;
        const float inv_l = seen ? 1.f / l : 0.f;
        const float lse2 = seen ? m + __log2f(l) : -INFINITY;
        const float c0 = a0 * inv_l, c1 = a1 * inv_l;
        // 32 columns at a time, the accumulators handed back to the PV issuer
        // behind the last.
        const TileUnit w = *unit;
        const bool boxed = O_BF16 && w.pieces == 1 && 32 * quad + 32 <= w.nq;
        store_lse(w, a, lse2, p.lse, p.part, p.args.T, D);
#pragma unroll 1
        for (int oc = 0; oc < D / 32; ++oc) {
          float ov[32];
          {
            uint32_t t0[32], t1[32];
            if (has0) {
              tmem_ld32(tmem + lane_base + kColO + par * D + oc * 32, t0);
              tmem_wait_ld(t0);
            }
            if (has1) {
              tmem_ld32(tmem + lane_base + kColO + (par ^ 1) * D + oc * 32, t1);
              tmem_wait_ld(t1);
            }
#pragma unroll
            for (int n = 0; n < 32; ++n)
              ov[n] = (has0 ? __uint_as_float(t0[n]) * c0 : 0.f) + (has1 ? __uint_as_float(t1[n]) * c1 : 0.f);
          }
          if (boxed) {
            // bf16 rows into this warp's quadrant of its own P buffer (free
            // until its next step: the last PV that read it is complete), then
            // one TMA store of the 32-row box, all of them the unit's.
            uint8_t* orow_s = sP + par * kQTile + (a / 8) * 1024 + (a % 8) * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(orow_s + (((4 * oc + c) ^ (a % 8)) * 16)) =
                  make_uint4(pack_bf16x2(ov[8 * c], ov[8 * c + 1]), pack_bf16x2(ov[8 * c + 2], ov[8 * c + 3]),
                             pack_bf16x2(ov[8 * c + 4], ov[8 * c + 5]), pack_bf16x2(ov[8 * c + 6], ov[8 * c + 7]));
          } else {
            store_columns<D, O_BF16>(w, a, oc, ov, p.o, p.part, p.args.H);
          }
        }
        warp_arrive_tc(&bars->o_free);
        if (boxed) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tm.o, sP + par * kQTile + quad * 4096, 0, w.h, w.row0 + 32 * quad);
            bulk_commit_group();
          }
          store_pending = true;
        }
      }
      if (!has_next) break;
      gt = g0 + nks;
      ++un;
      rb = (rb + nks + 2) & (kSlots - 1);
    }
    if (!ok) report_timeout(abort, p.args.status);
    // Output stores in flight must finish before the CTA's shared memory goes.
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }

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
  auto kern = paged_tc64_kernel<O_BF16, STALL>;
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

cudaError_t launch_paged_tc64(const TileMaps& m, const TileParams& p, bool o_bf16, int sms, cudaStream_t stream) {
  if (p.inject_stall) return o_bf16 ? launch<true, true>(m, p, sms, stream) : launch<false, true>(m, p, sms, stream);
  return o_bf16 ? launch<true, false>(m, p, sms, stream) : launch<false, false>(m, p, sms, stream);
}

}  // namespace txl
