// cached_tc.cu -- attention of a block's rows over the 8-bit cache (cached_tc_kernel.cuh).
#include "cached_tc_kernel.cuh"

namespace bdlm {

cudaError_t launch_cached_tc(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  return launch_tc<false>(m, p, st, launches);
}

}  // namespace bdlm
