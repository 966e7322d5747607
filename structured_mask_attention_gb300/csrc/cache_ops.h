// cache_ops.h -- parameters and launchers of the calls that write, weigh and
// evict the 8-bit cache.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"

namespace bdlm {

struct AppendParams {
  CacheDesc c;
  RowsDesc r;
  const void *K, *V;  // bf16 [T, Hkv, d]
  int32_t* lens_out;
  uint32_t* status;
};
cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t st, int* launches);

struct WeightsParams {
  CacheDesc c;
  RowsDesc r;
  AttnSplit sp;  // keyed
  const void* Q;     // bf16 [T, Hq, d]
  const float* LSE;  // [Hq, T]
  int Hq;
  float sl2;
  float* W;  // [n_seqs, Hkv, max_pages * page]
  int G;     // CTAs
  uint32_t* status;
  uint64_t limit_ns;
};
// k8: K's codes as [n_pages * Hkv, page, d].
cudaError_t launch_cache_weights(const CUtensorMap& k8, const WeightsParams& p, cudaStream_t st, int* launches);

struct EvictParams {
  CacheDesc c;
  const int32_t* dst;  // [n_seqs, max_pages]
  const float* W;      // [n_seqs, Hkv, max_pages * page]
  float* W_out;        // same shape
  int32_t* kept;       // [n_seqs, Hkv, keep]
  int32_t* lens_out;
  int keep, sinks, recent;
  uint32_t* status;
};
cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t st, int* launches);

}  // namespace bdlm
