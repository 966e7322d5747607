// cached_attn.h -- parameters and launchers of the attention over the 8-bit cache.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"

namespace bdlm {

struct CachedParams {
  CacheDesc c;
  RowsDesc r;
  AttnSplit sp;
  const void *Q, *K, *V;  // bf16 [T, Hq, d], [T, Hkv, d]
  int Hq;
  float sl2;  // softmax scale * log2(e)
  void* O;
  int o_f32;
  float* LSE;
  float* part;  // two partial results per CTA of G
  int G;
  uint32_t* status;
  uint64_t limit_ns;
};

// A partial result: O (not yet divided by the row sum) of tile_rows rows,
// then their running maxima (log2 units) and sums, all fp32.
__host__ __device__ inline int64_t part_floats(int tile_rows, int d) { return (int64_t)tile_rows * (d + 2); }

constexpr int kSmallRows = 16;       // row tile of the mma.sync kernel
constexpr int kSmallCtasPerSm = 2;   // its resident CTAs

cudaError_t launch_cached_small(const CachedParams& p, cudaStream_t st, int* launches);
cudaError_t launch_cached_merge(const CachedParams& p, cudaStream_t st, int* launches);

}  // namespace bdlm
