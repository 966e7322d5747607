// tree_tc.cu -- attention of the rows of drafted trees over the 8-bit cache:
// the kernel of cached_tc_kernel.cuh with visibility words.
#include "cached_tc_kernel.cuh"

namespace bdlm {

cudaError_t launch_tree_tc(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  return launch_tc<true>(m, p, st, launches);
}

}  // namespace bdlm
