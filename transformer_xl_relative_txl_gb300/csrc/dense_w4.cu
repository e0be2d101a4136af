// Products of a few rows with 4-bit weights: y = x W (+ bias) (ReLU),
//
//   W[j, i] = scales[j / G, i] * (code[i, j] - 8),   codes two to a byte along j
//
// Its floor is reading the codes once.  131072 columns of 1024 for 8 tokens take
// 19.4 us, 3.8 TB/s: a warp executes 24.8 instructions for each word of 8 codes, of
// which 9, by the source, make bf16 of them; the others are the products, x from
// shared memory for every 16 columns, the groups' sums, copies and their addresses.
// The schedulers issue in 66% of the active cycles and no pipe is over 51%, so that
// none alone is what bounds it.  Small products are a chain of launch, first blocks
// and sums: 512 x 512 for one token 3.0 us; 4096 x 1024 for 32 6.1, of whose 9200
// cycles, when nothing runs beside it, x takes 2200 (most of them the first load's
// way), the blocks of codes 2000 and the sums of the cluster's CTAs 4500.
//
// All instantiations for 16 and 32 tokens (128 registers) and that of groups of 64
// for 8 (80) spill, 12 to 28 bytes.
//
// The weights are the long operand, on the M side of mma.sync m16n8k16: a warp takes
// 16 of W's columns (n) by 256 rows (k) at a time, 2 KB of codes, which it brings to
// its own shared memory by cp.async, several blocks ahead, without any other warp's
// part.  The tokens are the 8 columns of the right-hand side, 8, 16 or 32 of them.
// (tcgen05 wants both operands in shared or tensor memory: the bf16 values of the
// codes would be stored and read once more, four times the codes' bytes, for tensor
// cores that are a fifth busy.)
//
// Nothing is rounded on the way: a code less 8 is exact in bf16 and so is x, the
// products are summed in fp32 over a group and the sum times the scale is added
// to the fp32 total.  (Both in units of 1 / 64, see below: exact, but for sums near
// 2^-126.)
//
// The low 8 bits of a bf16 number are its multiple of 2^-133, so a code, alone in
// the lower or upper four of them, becomes its value less 8, in units of 1 / 64, by
// one fma with 2^127 or 2^123, two codes at a time: codes c and c + 4 of a 32-bit
// word of 8.  (As 128 + code, less 136, it needs two shifts more for 8 codes: 21.1
// us against 19.4 for 131072 columns of 1024.)  The sum over k has no order, so x is
// laid out in shared memory by the same pairs, (0,4) (1,5) (2,6) (3,7) of every 8,
// and one ldmatrix hands each lane the words that it needs: lane (g, t) gets word t
// of chunk w of row g, codes 32 w + 8 t .. + 7, so that the 16 values of a step lie
// within one group of 32 or more.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "pdl.cuh"
#include "tokens.h"
#include "txl_device.cuh"

namespace cg = cooperative_groups;

namespace txl {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kBlockK = 256;               // codes of a row in a block: 128 bytes
constexpr int kCodeBytes = 16 * kBlockK / 2;
constexpr int kXBytes = 64 * 1024;         // of x in shared memory
constexpr int kMaxSplit = 8;

struct Args {
  const __nv_bfloat16* x;
  const uint8_t* codes;
  const __nv_bfloat16* scales;
  void* y;
  const float* bias;
  int m, n, k;
  int wr_log;  // 2^wr_log of the warps stand along n, the others share the blocks of k
  int split;   // CTAs of a cluster that share k
  int ks;      // rows of k of one of them, a multiple of kBlockK
  int kx;      // of these, rows whose x is in shared memory at a time, a multiple of kBlockK
  bool relu;
};

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Codes j and j + 4 of a word, less 8, times kUnit, as bf16.
constexpr float kUnit = 1.f / 64;
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
struct Codes {
  uint32_t at[4];
};
__device__ __forceinline__ Codes codes_of(uint32_t word) {
  const uint32_t upper = word >> 8;
  constexpr uint32_t kLo = 0x000F000Fu, kHi = 0x00F000F0u;        // the codes' places
  constexpr uint32_t kOfLo = 0x7F007F00u, kOfHi = 0x7D007D00u;    // 2^127 and 2^123
  constexpr uint32_t kLess = 0xBE00BE00u;                         // -8 / 64
  return Codes{{fma_bf16x2(word & kLo, kOfLo, kLess), fma_bf16x2(word & kHi, kOfHi, kLess),
                fma_bf16x2(upper & kLo, kOfLo, kLess), fma_bf16x2(upper & kHi, kOfHi, kLess)}};
}

template <int G, int MT>
struct Shape {
  static constexpr int kStages = MT == 1 ? 3 : 4;  // blocks of a warp, one less in flight
  static constexpr int kPerSm = MT == 1 ? 3 : 2;
  static constexpr int kGroups = kBlockK / G;  // of a block
  static constexpr int kScaleBytes = kGroups * 32;
  static constexpr int kStage = kCodeBytes + kScaleBytes;
  static constexpr int kTokens = 8 * MT;
  static constexpr int kPartBytes = kWarps * 16 * kTokens * 4;  // the warps' sums
  // A token's row of x: 8 lanes' 16-byte reads (two tokens, 64 bytes of each)
  // meet all banks where rows are 64 bytes off a multiple of 128.
  static constexpr int pitch(int kx) { return kx * 2 + 64; }
  static constexpr int smem(int kx) { return kWarps * kStages * kStage + kPartBytes + kTokens * pitch(kx); }
};

// Output i, from its sum.
template <bool YB>
__device__ __forceinline__ void put(const Args& p, size_t i, float v) {
  if (p.relu) v = v < 0.f ? 0.f : v;  // NaN stays
  if constexpr (YB) static_cast<__nv_bfloat16*>(p.y)[i] = __float2bfloat16(v);
  else static_cast<float*>(p.y)[i] = v;
}

// YB: y is bf16.  A CTA takes tiles of 16 * 2^wr_log columns of W and its part of
// k; a warp's blocks, of one tile after the other, are one line, of which the
// next kStages - 1 are always on their way.
template <int G, int MT, bool YB>
__global__ void __launch_bounds__(kThreads, Shape<G, MT>::kPerSm) dense_w4_kernel(const Args p) {
  using S = Shape<G, MT>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* stages = smem + warp * kStages * S::kStage;
  float* parts = reinterpret_cast<float*>(smem + kWarps * kStages * S::kStage);  // [warp][token][16]
  uint8_t* xs = smem + kWarps * kStages * S::kStage + S::kPartBytes;
  const int pitch = S::pitch(p.kx);
  const int wr = 1 << p.wr_log, wk = kWarps >> p.wr_log;
  const int my_r = warp & (wr - 1), my_k = warp >> p.wr_log;
  const int tiles = (p.n + 16 * wr - 1) / (16 * wr);
  const int rank = static_cast<int>(blockIdx.x) % p.split;
  const int tile0 = static_cast<int>(blockIdx.x) / p.split, tile_step = static_cast<int>(gridDim.x) / p.split;
  const int ka = rank * p.ks, ke = min(p.k, ka + p.ks);  // this CTA's rows of k
  const int blocks = ke > ka ? (ke - ka + kBlockK - 1) / kBlockK : 0;
  const int tok0 = static_cast<int>(blockIdx.y) * S::kTokens;
  const int tokens = min(S::kTokens, p.m - tok0);
  const int g = lane >> 2, t = lane & 3;
  if (p.split > 1) cg::this_cluster().barrier_arrive();
  grid_dep_wait();
  grid_dep_launch_dependents();

  // The line of this warp's blocks: where the copies are.  A lane copies chunk
  // lane % 8 of rows lane / 8, + 4, + 8 and + 12, and, of some lanes, 8 scales.
  int f_tile = tile0, f_block = my_k, f_slot = 0;
  const uint32_t to = smem_u32(stages) + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
  const uint32_t to_odd = smem_u32(stages) + (lane >> 3) * 128 + (((lane & 7) ^ (4 + (lane >> 3))) << 4);
  const size_t row_bytes = static_cast<size_t>(p.k) / 2, rows4 = 4 * row_bytes;
  const uint8_t* from;
  const __nv_bfloat16* from_s;
  bool whole;  // no row of the tile past the end
  const auto place = [&]() {
    const int n0 = (f_tile * wr + my_r) * 16, kb = ka + f_block * kBlockK;
    from = p.codes + (n0 + (lane >> 3)) * row_bytes + kb / 2 + (lane & 7) * 16;
    from_s = p.scales + static_cast<size_t>(kb / G + (lane >> 1)) * p.n + n0 + (lane & 1) * 8;
    whole = n0 + 16 <= p.n;
  };
  if (f_block < blocks) place();
  const auto fetch = [&]() {
    if (f_tile < tiles && f_block < blocks) {
      const uint32_t at = f_slot * S::kStage;
      const int kb = ka + f_block * kBlockK;
      if (whole && kb + kBlockK <= ke) {
        copy16(to + at, from, true);
        copy16(to_odd + at + 4 * 128, from + rows4, true);
        copy16(to + at + 8 * 128, from + 2 * rows4, true);
        copy16(to_odd + at + 12 * 128, from + 3 * rows4, true);
        if (lane < 2 * S::kGroups) copy16(smem_u32(stages) + at + kCodeBytes + lane * 16, from_s, true);
      } else {
        const int n0 = (f_tile * wr + my_r) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool there = n0 + i * 4 + (lane >> 3) < p.n && kb + (lane & 7) * 32 < ke;
          copy16((i & 1 ? to_odd : to) + at + i * 512, there ? from + i * rows4 : p.codes, there);
        }
        if (lane < 2 * S::kGroups) {
          const bool there = kb + (lane >> 1) * G < ke && n0 + (lane & 1) * 8 < p.n;
          copy16(smem_u32(stages) + at + kCodeBytes + lane * 16, there ? from_s : p.scales, there);
        }
      }
      f_block += wk;
      from += wk * (kBlockK / 2);
      from_s += static_cast<size_t>(wk * S::kGroups) * p.n;
      if (f_block >= blocks) {
        f_block = my_k, f_tile += tile_step;
        if (f_tile < tiles) place();
      }
    }
    copies_commit();
    f_slot = f_slot == kStages - 1 ? 0 : f_slot + 1;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch();

  int slot = 0;
  for (int tile = tile0; tile < tiles; tile += tile_step) {
    const int n0 = (tile * wr + my_r) * 16;
    float total[MT][4];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) total[a][e] = 0.f;
    for (int k0 = ka; k0 < ke; k0 += p.kx) {
      const int k1 = min(ke, k0 + p.kx);
      if (p.ks > p.kx || tile == tile0) {
        // x of this stretch, by pairs; zeros past its end.
        if (p.ks > p.kx) __syncthreads();
        const int octets = (k1 - k0 + kBlockK - 1) / kBlockK * (kBlockK / 8);  // of a token, a multiple of 32
        // Warp w takes tokens w, w + 8, ...: eight of a lane's copies at a time.
        const int there = (k1 - k0) / 8;
        const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(tok0 + warp) * p.k + k0);
        for (int o = lane; o < octets; o += 256 / MT) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int a = i % MT, at = o + i / MT * 32;
            v[i] = make_uint4(0, 0, 0, 0);
            if (warp + 8 * a < tokens && at < there) v[i] = __ldg(src + static_cast<size_t>(a) * p.k + at);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int a = i % MT, at = o + i / MT * 32;
            if (at < octets)
              *reinterpret_cast<uint4*>(xs + (warp + 8 * a) * pitch + at * 16) =
                  make_uint4(__byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                             __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
          }
        }
        __syncthreads();
      }
      // This warp's blocks of the stretch.
      const int b0 = (k0 - ka) / kBlockK, b1 = (k1 - ka + kBlockK - 1) / kBlockK;
      for (int b = b0 + ((my_k - b0) & (wk - 1)); b < b1; b += wk) {
        copies_wait<kStages - 2>();
        __syncwarp();  // every lane's copies are there, and all have read the slot that is filled next
        fetch();
        const uint8_t* at = stages + slot * S::kStage;
        const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(at + kCodeBytes);
        const uint8_t* xb = xs + g * pitch + ((b - b0) * kBlockK + t * 8) * 2;
        // Two sums at a time for a single column of tokens: the products of one wait for each other.
        constexpr int kSums = MT == 1 ? 2 : 1;
        float acc[kSums][MT][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = lane & 7, chunk = half * 4 + (lane >> 3);
          const uint32_t from = smem_u32(at) + row * 128 + ((chunk ^ row) << 4);
          uint32_t lo[4], hi[4];
          ldsm4(from, lo);
          ldsm4(from + 8 * 128, hi);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int c = half * 4 + w;  // chunk of 32 codes
            if (c % (G / 32) == 0) {
#pragma unroll
              for (int s = 0; s < kSums; ++s)
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[s][a][e] = 0.f;
            }
            const Codes l = codes_of(lo[w]), h = codes_of(hi[w]);
            const uint32_t wa[4] = {l.at[0], h.at[0], l.at[1], h.at[1]};
            const uint32_t wb[4] = {l.at[2], h.at[2], l.at[3], h.at[3]};
#pragma unroll
            for (int a = 0; a < MT; ++a) {
              const uint4 v = *reinterpret_cast<const uint4*>(xb + a * 8 * pitch + c * 64);
              mma16816(acc[0][a], wa, v.x, v.y);
              mma16816(acc[kSums - 1][a], wb, v.z, v.w);
            }
            if ((c + 1) % (G / 32) == 0) {
              const int group = c / (G / 32);
              const float s0 = __bfloat162float(sc[group * 16 + g]), s1 = __bfloat162float(sc[group * 16 + g + 8]);
#pragma unroll
              for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float sum = kSums == 2 ? acc[0][a][e] + acc[kSums - 1][a][e] : acc[0][a][e];
                  total[a][e] = fmaf(sum, e < 2 ? s0 : s1, total[a][e]);
                }
            }
          }
        }
        slot = slot == kStages - 1 ? 0 : slot + 1;
      }
    }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) total[a][e] *= 1.f / kUnit;
    if (wk == 1 && p.split == 1) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int col = n0 + g + 8 * r;
        if (col >= p.n) continue;
        const float bias = p.bias != nullptr ? __ldg(p.bias + col) : 0.f;
        size_t i = static_cast<size_t>(tok0 + 2 * t) * p.n + col;
#pragma unroll
        for (int a = 0; a < MT; ++a, i += 8 * static_cast<size_t>(p.n)) {
          if (a * 8 + 2 * t < tokens) put<YB>(p, i, total[a][2 * r] + bias);
          if (a * 8 + 2 * t + 1 < tokens) put<YB>(p, i + p.n, total[a][2 * r + 1] + bias);
        }
      }
      continue;
    }
    // The warps, and the CTAs, that shared k add up, in order: the sums go to
    // shared memory, and each CTA of the cluster takes its share of the outputs.
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        parts[(warp * S::kTokens + a * 8 + 2 * t + (e & 1)) * 16 + g + 8 * (e >> 1)] = total[a][e];
    const int cols_log = 4 + p.wr_log, outs = tokens << cols_log;
    const auto place_of = [&](int o) {
      const int token = o >> cols_log, c = o & ((1 << cols_log) - 1);
      return ((c >> 4) * S::kTokens + token) * 16 + (c & 15);
    };
    const auto finish = [&](int o, float v) {
      const int col = tile * 16 * wr + (o & ((1 << cols_log) - 1));
      if (col >= p.n) return;
      if (p.bias != nullptr) v += __ldg(p.bias + col);
      put<YB>(p, static_cast<size_t>(tok0 + (o >> cols_log)) * p.n + col, v);
    };
    const int warp_part = wr * S::kTokens * 16;  // from one warp's sums to those of the next that shares its columns
    __syncthreads();
    if (p.split == 1) {
      for (int o = threadIdx.x; o < outs; o += kThreads) {
        const int at = place_of(o);
        float v = parts[at];
        for (int w = 1; w < wk; ++w) v += parts[w * warp_part + at];
        finish(o, v);
      }
      __syncthreads();
      continue;
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (wk > 1) {
      for (int o = threadIdx.x; o < outs; o += kThreads) {
        const int at = place_of(o);
        float v = parts[at];
        for (int w = 1; w < wk; ++w) v += parts[w * warp_part + at];
        parts[at] = v;
      }
    }
    if (tile == tile0) cluster.barrier_wait();
    cluster.sync();
    const int o1 = outs * (rank + 1) / p.split;
    for (int o = outs * rank / p.split + static_cast<int>(threadIdx.x); o < o1; o += kThreads) {
      float part[kMaxSplit];  // all on their way together
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        part[r] = r < p.split ? cluster.map_shared_rank(parts, r)[place_of(o)] : 0.f;
      float v = part[0];
#pragma unroll
      for (int r = 1; r < kMaxSplit; ++r) v += part[r];
      finish(o, v);
    }
    cluster.sync();
  }
  copies_wait<0>();
}

template <int G, int MT, bool YB>
cudaError_t launch(Args a, cudaStream_t stream) {
  using S = Shape<G, MT>;
  constexpr int kMaxX = kXBytes / (2 * S::kTokens) / kBlockK * kBlockK;
  const int blocks = (a.k + kBlockK - 1) / kBlockK;
  // How many warps stand along n and how many CTAs share k, by the time that a
  // pair takes: fitted to 250 measured ones (m 1 to 32, k 128 to 8192, n 512 to
  // 131072), whose best it misses by 12% at most.  In ns: each block of the SM with
  // the most, a sum of warps, of CTAs, 1 KB of x.  Both ends: 32 tokens, k =
  // 4096, n = 1024 take 21 us with a CTA for 128 columns and all of k, 6.3 with a
  // cluster of four for 32; 8 tokens, k = 1024, n = 131072 take 19.4 with the first
  // and 98 with a cluster of four for 64.  (Fitted with fewer clusters of 8 at a
  // time than there is room for, 12, 24 and 36, and more of 4, 38, 76 and 114; where
  // that decides, the true counts give: 8 tokens, k = 8192, n = 5792 10.4 us for
  // 14.2, 16 tokens, 8192, 23168 41 for 62, 16 tokens, 8192, 4096 10.5 for 10.2.)
  // It plans for one block of tokens: of more than 32 rows each block of 32 has such
  // a grid, side by side (64 rows, k = 1024, n = 4096 take 8.5 us, 512 56).
  constexpr int kEach = MT == 1 ? 70 : MT == 2 ? 90 : 190;
  long long best = -1;
  int best_clusters = 1, best_smem = 0;
  for (int wr_log = 3; wr_log >= 0; --wr_log)
    for (int log = 0, split = 1; split <= kMaxSplit && (split == 1 || split <= blocks); split = 1 << ++log) {
      const int tiles = (a.n + (16 << wr_log) - 1) / (16 << wr_log), wk = kWarps >> wr_log;
      const int mine = (blocks + split - 1) / split, kx = std::min(mine * kBlockK, kMaxX);
      const int smem = S::smem(kx);
      const int per_sm = std::max(1, std::min(S::kPerSm, 227 * 1024 / (smem + 1024)));
      const int clusters = std::min(tiles, clusters_at_a_time(log, per_sm));
      const long long rounds = (tiles + clusters - 1) / clusters;
      const long long on_sm = (static_cast<long long>(tiles) * split + 151) / 152 * mine << wr_log;  // blocks
      const long long ns = on_sm * kEach + rounds * ((wk > 1 ? 670 : 0) + (split > 1 ? 2100 : 0)) +
                           8LL * mine * kBlockK * S::kTokens * 2 / 1024 * (mine * kBlockK > kMaxX ? rounds : 1);
      if (best >= 0 && ns >= best) continue;
      best = ns, best_clusters = clusters, best_smem = smem;
      a.wr_log = wr_log, a.split = split, a.ks = mine * kBlockK, a.kx = kx;
    }
  auto kernel = dense_w4_kernel<G, MT, YB>;
  // The most that any call needs: another thread may set it at the same time.
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem(kMaxX));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(best_clusters * a.split, (a.m + S::kTokens - 1) / S::kTokens);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = best_smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int G, bool YB>
cudaError_t by_tokens(const Args& a, cudaStream_t stream) {
  if (a.m <= 8) return launch<G, 1, YB>(a, stream);
  if (a.m <= 16) return launch<G, 2, YB>(a, stream);
  return launch<G, 4, YB>(a, stream);
}

template <bool YB>
cudaError_t by_group(const Args& a, int group, cudaStream_t stream) {
  switch (group) {
    case 32: return by_tokens<32, YB>(a, stream);
    case 64: return by_tokens<64, YB>(a, stream);
    case 128: return by_tokens<128, YB>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_dense_w4(const void* x, const unsigned char* codes, const void* scales, void* y, const float* bias,
                            int m, int n, int k, int group, bool relu, bool y_bf16, cudaStream_t stream) {
  Args a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.codes = codes;
  a.scales = static_cast<const __nv_bfloat16*>(scales);
  a.y = y;
  a.bias = bias;
  a.m = m, a.n = n, a.k = k;
  a.relu = relu;
  return y_bf16 ? by_group<true>(a, group, stream) : by_group<false>(a, group, stream);
}

}  // namespace txl
