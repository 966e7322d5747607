// tree_small.cu -- attention of up to 32 rows of drafted trees over the 8-bit cache:
// the kernel of cached_small.cuh with visibility words.
#include "cached_small.cuh"

namespace bdlm {

cudaError_t launch_tree_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  return launch_small<true>(m, p, st, launches);
}

}  // namespace bdlm
