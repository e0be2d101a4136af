// Internal interface of the operators around the layers (embed.cu,
// dense_w4.cu, sample.cu) to their C entry points (tokens_api.cu).  Arguments
// are validated by the caller.
#pragma once

#include <cuda_runtime.h>

namespace txl {

// How many clusters of 2^log CTAs, of which an SM has room for per_sm, run at a
// time: cudaOccupancyMaxActiveClusters' answers for the products' and the sampler's
// kernels, which depend on per_sm alone.  A cluster stays within one group of SMs,
// so that those of 4 and 8 leave some idle.
inline int clusters_at_a_time(int log, int per_sm) {
  constexpr int kAt[3][4] = {{152, 76, 36, 15}, {304, 152, 74, 36}, {456, 228, 110, 51}};
  return kAt[per_sm - 1][log];
}

constexpr int kEmbedMaxRows = 1 << 24;    // rows of an embedding table
constexpr int kSampleMaxVocab = 1 << 18;  // logits of a row: its weights' sum fits 64 bits

cudaError_t launch_embed_forward(const int* tokens, const void* table, void* out, int T, int V, int d, float scale,
                                 bool table_bf16, bool out_bf16, cudaStream_t stream);
cudaError_t launch_embed_backward(const int* tokens, const void* dout, float* dtable, int T, int V, int d, float scale,
                                  bool accumulate, bool dout_bf16, cudaStream_t stream);

// codes 16-byte aligned, k a multiple of group, group 32, 64 or 128, n of 8.
cudaError_t launch_dense_w4(const void* x, const unsigned char* codes, const void* scales, void* y, const float* bias,
                            int m, int n, int k, int group, bool relu, bool y_bf16, cudaStream_t stream);

struct SampleArgs {
  const void* logits;
  long long row_stride;  // elements
  int B, V;
  const float* uniform;
  const float* temperature;  // this and the next three: nullptr where off for every row
  const int* top_k;
  const float* top_p;
  const float* min_p;
  int* tokens;
  float* prob;  // or nullptr
  bool bf16;
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream);

}  // namespace txl
