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
  int whole;    // not 0: a CTA per segment, that many row tiles for each (sequence, KV head)
  uint32_t* status;
  uint64_t limit_ns;
};

// A partial result, fp32: O (not yet divided by the row sum), four columns of
// all tile_rows rows together (so that threads that hold a row each write
// side by side), then the rows' reference maxima (log2 units) and sums.
__host__ __device__ inline int64_t part_floats(int tile_rows, int d) { return (int64_t)tile_rows * (d + 2); }

// Rows up to which the mma.sync kernel takes a call.  16 sequences of 16384
// tokens with 20 / 32 rows: 111 / 116 us here, 130 / 130 in the tcgen05
// kernel; 64 rows (16 sequences of 8192): 118 us here, 88 there.
constexpr int kSmallRows = 32;
constexpr int kSmallCtasPerSm = 2;  // its resident CTAs

// Row tile of a call whose sequences have at most `flat` rows times heads of
// a group: 16 or 32 (mma.sync), 128 or 256 (tcgen05, split and pairs).  Split
// serves any number of rows in tiles of 128; pairs read the keys half as often
// but hold 256 rows: split against pairs 82 / 83 us at 128 rows, 106 / 111 at
// 160, 92 / 84 at 256 (8 sequences of 8192), 174 / 177 at 384, 250 / 226 at 640,
// 537 / 487 at 1024.
inline int cached_tile_rows(int64_t flat) {
  return flat <= 16 ? 16 : flat <= kSmallRows ? 32 : flat <= 128 ? 128 : 256;
}
inline int cached_ctas(int tile_rows, int sms) { return tile_rows <= kSmallRows ? sms * kSmallCtasPerSm : sms; }

// Tensor maps: the codes as [n_pages * Hkv, page, d] (V's for the mma.sync
// kernel), the new rows' K and V as [T, Hkv, d] bf16 (for the tcgen05 kernel).
struct CachedMaps {
  CUtensorMap k8, v8, k, v;
};
cudaError_t launch_cached_tc(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches);
// Longest cache, in tokens, up to which the mma.sync kernel gives each segment
// one CTA: no work list to walk and no merge kernel, whose launch alone is about
// 4 us, against the four units of 128 keys, 0.7 us each, that it would share out.
constexpr int kWholeKeys = 1024;
// AttnSplit::extra: what a segment costs beside its units, in units.  The
// tcgen05 kernels spend 16 to 20 thousand cycles to begin and end a segment and
// 2060 (split) or 4150 (pairs) on a unit; with 0 / 6, blocks of 32 and 128 took
// 130 / 106 and 293 / 248 us.
constexpr int kSmallExtra = 3, kSmallExtraOwn = 5, kTcExtra = 6;

cudaError_t launch_cached_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches);
cudaError_t launch_cached_merge(const CachedParams& p, cudaStream_t st, int* launches);

}  // namespace bdlm
