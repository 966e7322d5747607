// tree_small.cu -- attention of few rows of drafted trees over the 8-bit cache:
// the kernel of cached_small.cuh with visibility words.
#include "cached_small.cuh"

namespace bdlm {

template <int HD, bool FINE>
static cudaError_t launch_rows(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  if (p.sp.tile_rows == 16) return launch<HD, 1, 1, FINE, true>(m, p, st);
  // 32 rows: both row tiles to each warp, which turns a key's codes into fp16 once for both, where the caches may be
  // long enough to pay for the larger beginning: from kBothUnits units to a CTA on.  A row tile to each of two warps
  // against both to each, chains of 5 over 32 sequences, 32 / 8 heads of 128: 50 / 53 us at 2048 tokens at most,
  // 73 / 71 at 4096, 114 / 108 at 8192, 198 / 173 at 16384, 363 / 299 at 32768; over 4 sequences 48 / 49 at 16384, 118 /
  // 110 at 65536; d = 64, 32 sequences: 49 / 45 at 4096, 135 / 115 at 16384.  (16 keys at a time instead of 32: 364
  // where 299; 64 rows this way, 32 to a warp: 104 us for 64 rows of 16 sequences where the tcgen05 kernel takes 86.)
  // fp32 outputs of 128 columns, whose two parts of P leave it no registers: 470 / 479.
  constexpr int64_t kBothUnits = 24;
  const int64_t units = (int64_t)p.c.n_seqs * p.c.Hkv * (((int64_t)p.c.max_pages * p.c.page + kUnit - 1) / kUnit);
  if constexpr (HD == 64 || !FINE)
    if (units >= kBothUnits * p.G) return launch<HD, 2, 1, FINE, true>(m, p, st);
  return launch<HD, 1, 2, FINE, true>(m, p, st);
}

cudaError_t launch_tree_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  const cudaError_t e = p.c.d == 128 ? (p.o_f32 ? launch_rows<128, true>(m, p, st) : launch_rows<128, false>(m, p, st))
                                     : (p.o_f32 ? launch_rows<64, true>(m, p, st) : launch_rows<64, false>(m, p, st));
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace bdlm
