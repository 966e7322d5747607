// tree_small.cu -- attention of few rows of drafted trees over the 8-bit cache:
// the kernel of cached_small.cuh with visibility words.
#include "cached_small.cuh"

namespace bdlm {

template <int HD, bool FINE>
static cudaError_t launch_rows(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  // 32 rows: both row tiles to each warp, which turns a key's codes into fp16 once for both (chains of 5 over 32
  // sequences of up to 32768 tokens, 32 / 8 heads of 128: 299 us; a row tile to each of two warps: 364; both tiles
  // and 16 keys at a time: 364.  64 rows this way, 32 to a warp: 104 us where the tcgen05 kernel takes 86.)
  return p.sp.tile_rows == 16 ? launch<HD, 1, 1, FINE, true>(m, p, st) : launch<HD, 2, 1, FINE, true>(m, p, st);
}

cudaError_t launch_tree_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  const cudaError_t e = p.c.d == 128 ? (p.o_f32 ? launch_rows<128, true>(m, p, st) : launch_rows<128, false>(m, p, st))
                                     : (p.o_f32 ? launch_rows<64, true>(m, p, st) : launch_rows<64, false>(m, p, st));
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace bdlm
