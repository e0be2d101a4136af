// Products of a few rows with 4-bit weights: y = x W (+ bias) (ReLU),
//
//   W[j, i] = scales[j / G, i] * (code[i, j] - 8),   codes two to a byte along j
//
// Bound by reading the codes once.  The weights are the long operand, on the M
// side of mma.sync m16n8k16: a warp takes 16 of W's columns (n) by 256 rows (k)
// at a time, 2 KB of codes, which it brings to its own shared memory by
// cp.async, several blocks ahead, without any other warp's part.  The tokens
// are the 8 columns of the right-hand side, 8, 16 or 32 of them.
//
// Nothing is rounded on the way: a code less 8 is exact in bf16 and so is x, the
// products are summed in fp32 over a group and the sum times the scale is added
// to the fp32 total.
//
// A code becomes a bf16 value by 0x4300 | code = 128 + code, less 136, two at a
// time: codes c and c + 4 of a 32-bit word of 8.  The sum over k has no order,
// so x is laid out in shared memory by the same pairs, (0,4) (1,5) (2,6) (3,7) of
// every 8, and one ldmatrix hands each lane the words that it needs: lane (g,
// t) gets word t of chunk w of row g, codes 32 w + 8 t .. + 7, so that the 16
// values of a step lie within one group of 32 or more.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "pdl.cuh"
#include "tokens.h"
#include "txl_device.cuh"

namespace txl {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kBlockK = 256;               // codes of a row in a block: 128 bytes
constexpr int kStages = 4;                 // blocks in flight per warp
constexpr int kCodeBytes = 16 * kBlockK / 2;
constexpr int kXBytes = 64 * 1024;         // of x in shared memory

struct Args {
  const __nv_bfloat16* x;
  const uint8_t* codes;
  const __nv_bfloat16* scales;
  void* y;
  const float* bias;
  int m, n, k;
  int wr_log;  // 2^wr_log of the warps stand along n, the others share the blocks of k
  int kx;      // rows of k whose x is in shared memory at a time, a multiple of kBlockK
  bool relu;
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Codes j and j + 4 of a word, less 8, as bf16.
template <int J>
__device__ __forceinline__ uint32_t pair_of(uint32_t word) {
  const uint32_t w = (word >> (4 * J) & 0x000F000Fu) | 0x43004300u;
  const uint32_t less = 0xC308C308u;  // -136
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(less));
  return r;
}

template <int G, int MT>
struct Shape {
  static constexpr int kGroups = kBlockK / G;  // of a block
  static constexpr int kScaleBytes = kGroups * 32;
  static constexpr int kStage = kCodeBytes + kScaleBytes;
  static constexpr int kTokens = 8 * MT;
  // A token's row of x: 8 lanes' 16-byte reads (two tokens, 64 bytes of each)
  // meet all banks where rows are 64 bytes off a multiple of 128.
  static constexpr int pitch(int kx) { return kx * 2 + 64; }
  static constexpr int smem(int kx) { return kWarps * kStages * kStage + kTokens * pitch(kx); }
};

// YB: y is bf16.
template <int G, int MT, bool YB>
__global__ void __launch_bounds__(kThreads, 1) dense_w4_kernel(const Args p) {
  using S = Shape<G, MT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* stages = smem + warp * kStages * S::kStage;
  uint8_t* xs = smem + kWarps * kStages * S::kStage;
  const int pitch = S::pitch(p.kx);
  const int wr = 1 << p.wr_log, wk = kWarps >> p.wr_log;
  const int my_r = warp & (wr - 1), my_k = warp >> p.wr_log;
  const int tiles = (p.n + 16 * wr - 1) / (16 * wr);
  const int tok0 = static_cast<int>(blockIdx.y) * S::kTokens;
  const int tokens = min(S::kTokens, p.m - tok0);
  const int g = lane >> 2, t = lane & 3;
  grid_dep_wait();
  grid_dep_launch_dependents();

  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int n0 = (tile * wr + my_r) * 16;
    float total[MT][4];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) total[a][e] = 0.f;
    for (int k0 = 0; k0 < p.k; k0 += p.kx) {
      const int k1 = min(p.k, k0 + p.kx);
      const int blocks = (k1 - k0 + kBlockK - 1) / kBlockK;
      // Blocks my_k, my_k + wk, ... of this stretch of k.
      const auto fetch = [&](int b, int slot) {
        if (b < blocks) {
          uint8_t* at = stages + slot * S::kStage;
          const int kb = k0 + b * kBlockK;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = i * 4 + (lane >> 3), chunk = lane & 7;
            const bool there = n0 + row < p.n && kb + chunk * 32 < k1;
            const uint8_t* src = p.codes;
            if (there) src += static_cast<size_t>(n0 + row) * (p.k / 2) + kb / 2 + chunk * 16;
            copy16(at + row * 128 + ((chunk ^ (row & 7)) << 4), src, there);
          }
          if (lane < 2 * S::kGroups) {
            const int group = kb / G + (lane >> 1), col = n0 + (lane & 1) * 8;
            const bool there = group < p.k / G && col < p.n;
            const __nv_bfloat16* src = p.scales;
            if (there) src += static_cast<size_t>(group) * p.n + col;
            copy16(at + kCodeBytes + lane * 16, src, there);
          }
        }
        copies_commit();
      };
#pragma unroll
      for (int s = 0; s < kStages - 1; ++s) fetch(my_k + s * wk, s);
      if (p.k > p.kx || tile == static_cast<int>(blockIdx.x)) {
        // x of this stretch, by pairs; zeros past its end.
        if (p.k > p.kx) __syncthreads();
        const int octets = blocks * (kBlockK / 8);
        for (int i = threadIdx.x; i < S::kTokens * octets; i += kThreads) {
          const int row = i / octets, o = i - row * octets;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (row < tokens && k0 + o * 8 < k1)
            v = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(tok0 + row) * p.k + k0 + o * 8));
          uint4 w;
          w.x = __byte_perm(v.x, v.z, 0x5410);
          w.y = __byte_perm(v.x, v.z, 0x7632);
          w.z = __byte_perm(v.y, v.w, 0x5410);
          w.w = __byte_perm(v.y, v.w, 0x7632);
          *reinterpret_cast<uint4*>(xs + row * pitch + o * 16) = w;
        }
        __syncthreads();
      }
      int slot = 0;
      for (int b = my_k; b < blocks; b += wk) {
        copies_wait<kStages - 2>();
        __syncwarp();  // every lane's copies are there, and all have read the slot that is filled next
        fetch(b + (kStages - 1) * wk, slot == 0 ? kStages - 1 : slot - 1);
        const uint8_t* at = stages + slot * S::kStage;
        const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(at + kCodeBytes);
        const uint8_t* xb = xs + g * pitch + (b * kBlockK + t * 8) * 2;
        float acc[MT][4];
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
              for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[a][e] = 0.f;
            }
            const uint32_t wa[4] = {pair_of<0>(lo[w]), pair_of<0>(hi[w]), pair_of<1>(lo[w]), pair_of<1>(hi[w])};
            const uint32_t wb[4] = {pair_of<2>(lo[w]), pair_of<2>(hi[w]), pair_of<3>(lo[w]), pair_of<3>(hi[w])};
#pragma unroll
            for (int a = 0; a < MT; ++a) {
              const uint4 v = *reinterpret_cast<const uint4*>(xb + a * 8 * pitch + c * 64);
              mma16816(acc[a], wa, v.x, v.y);
              mma16816(acc[a], wb, v.z, v.w);
            }
            if ((c + 1) % (G / 32) == 0) {
              const int group = c / (G / 32);
              const float s0 = __bfloat162float(sc[group * 16 + g]), s1 = __bfloat162float(sc[group * 16 + g + 8]);
#pragma unroll
              for (int a = 0; a < MT; ++a) {
                total[a][0] = fmaf(acc[a][0], s0, total[a][0]);
                total[a][1] = fmaf(acc[a][1], s0, total[a][1]);
                total[a][2] = fmaf(acc[a][2], s1, total[a][2]);
                total[a][3] = fmaf(acc[a][3], s1, total[a][3]);
              }
            }
          }
        }
        slot = slot == kStages - 1 ? 0 : slot + 1;
      }
      copies_wait<0>();
      __syncwarp();
    }
    // The warps that shared k add up, in order, over the first one's stages.
    if (wk > 1) {
      float* parts = reinterpret_cast<float*>(stages);
      __syncthreads();
      if (my_k > 0) {
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) parts[(a * 4 + e) * 32 + lane] = total[a][e];
      }
      __syncthreads();
      if (my_k == 0) {
        for (int w = 1; w < wk; ++w) {
          const float* from = reinterpret_cast<const float*>(smem + (warp + w * wr) * kStages * S::kStage);
#pragma unroll
          for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) total[a][e] += from[(a * 4 + e) * 32 + lane];
        }
      }
      __syncthreads();
    }
    if (my_k == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int col = n0 + g + 8 * r;
        if (col >= p.n) continue;
        const float b = p.bias != nullptr ? __ldg(p.bias + col) : 0.f;
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int token = a * 8 + 2 * t + e;
            if (token >= tokens) continue;
            float v = total[a][2 * r + e] + b;
            if (p.relu) v = v < 0.f ? 0.f : v;  // NaN stays
            const size_t i = static_cast<size_t>(tok0 + token) * p.n + col;
            if constexpr (YB) static_cast<__nv_bfloat16*>(p.y)[i] = __float2bfloat16(v);
            else static_cast<float*>(p.y)[i] = v;
          }
      }
    }
  }
}

template <int G, int MT, bool YB>
cudaError_t launch(Args a, cudaStream_t stream) {
  using S = Shape<G, MT>;
  a.kx = std::min((a.k + kBlockK - 1) / kBlockK * kBlockK, kXBytes / (2 * S::kTokens) / kBlockK * kBlockK);
  // As many warps along n as leave a tile for every SM.
  a.wr_log = 3;
  while (a.wr_log > 0 && (a.n + (16 << a.wr_log) - 1) / (16 << a.wr_log) < 152) --a.wr_log;
  const int tiles = (a.n + (16 << a.wr_log) - 1) / (16 << a.wr_log);
  const int smem = S::smem(a.kx);
  auto kernel = dense_w4_kernel<G, MT, YB>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int per_sm = std::max(1, std::min(8, 227 * 1024 / (smem + 1024)));
  const dim3 grid(std::min(tiles, 152 * per_sm), (a.m + S::kTokens - 1) / S::kTokens);
  return launch_dependent(kernel, grid, dim3(kThreads), smem, stream, a);
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
  const Args a{static_cast<const __nv_bfloat16*>(x), codes, static_cast<const __nv_bfloat16*>(scales), y, bias, m, n,
               k, 0, 0, relu};
  return y_bf16 ? by_group<true>(a, group, stream) : by_group<false>(a, group, stream);
}

}  // namespace txl
