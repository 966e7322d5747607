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
  const uint32_t* vis;  // (trees) [T, words]: bit j % 32 of word j / 32: the row sees row j of its sequence
  int words;
  void* O;
  int o_f32;
  float* LSE;
  float* part;  // two partial results per CTA of G
  float* fine;  // (fp32 outputs, tcgen05) behind them: two sub-tiles' sums, 128 x d, per CTA
  int G;
  int whole;    // not 0: a CTA per segment, that many row tiles for each (sequence, KV head)
  uint32_t* status;
  uint64_t limit_ns;
};

// A partial result, fp32: O (not yet divided by the row sum), four columns of
// all tile_rows rows together (so that threads that hold a row each write
// side by side), then the rows' reference maxima (log2 units) and sums.
__host__ __device__ inline int64_t part_floats(int tile_rows, int d) { return (int64_t)tile_rows * (d + 2); }

// Rows up to which the mma.sync kernels take a call.  16 sequences of up to 16384
// tokens with 20 / 32 rows: 108 / 108 us here, 128 / 127 in the tcgen05 kernel (in a
// graph, warm); 64 rows (16 sequences of up to 8192): 118 us with tiles of 64 rows
// here, when it was tried, 83 there (trees: 92 in two tiles of 32 of tree_small.cu, 80 there).
constexpr int kSmallRows = 32;
constexpr int kSmallCtasPerSm = 2;  // its resident CTAs
// Weights are kept in fp16, 2^shift larger than exp2(s - reference): the largest
// come near 2^16, its end, and its range lies below them.  cached_small.cu has
// the exact running maximum for a reference: a weight keeps 11 bits down to 2^-29
// of the row's largest and counts down to 2^-40 (tree_small.cu: one bit less).  The tcgen05 kernels' reference
// may lie kRescale behind the maximum (and a tenth of a bit for rounding): 11
// bits down to 2^-23 of the reference, something down to 2^-34.  Such weights make up O
// where one key dominates a row and has a small value, an attention sink.  The
// rarer the rescaling, the less range: steps of 8 / 7 / 6 / 5 / 4 took 87.0 / 87.3 / 88.2 /
// 89.6 / 90.5 us for blocks of 32 and 225 / 228 / 229 / 231 / 232 for blocks of 128; 512
// were level.  The row sum takes p' 2^-shift.  (Scores so large that their rounding
// exceeds the margin: the exact maximum's shift is rounded up, p' saturates.)
constexpr float kRescale = 6.9f;  // log2 units: the tcgen05 kernels' reference moves in steps of at least this
constexpr float kSmallShift = 15.0f, kTcShift = 9.0f;
constexpr float kSmallUnshift = 1.0f / (1 << (int)kSmallShift), kTcUnshift = 1.0f / (1 << (int)kTcShift);

// Row tile of a call whose sequences have at most `flat` rows times heads of
// a group: 16 or 32 (mma.sync), 128 or 256 (tcgen05, split and pairs).  Split
// could serve any number of rows in tiles of 128; pairs read the keys half as
// often but hold 256 rows.  Split against pairs (8 sequences of up to 8192, in a
// graph, warm): 69 / 73 us at 160 rows, 79 / 78 at 256, 123 / 117 at 384, 213 / 188 at
// 640, 374 / 260 at 1024.
inline int cached_tile_rows(int64_t flat) {
  return flat <= 16 ? 16 : flat <= kSmallRows ? 32 : flat <= 128 ? 128 : 256;
}
// Trees: 257 to 384 rows go in three tiles of 128; of pairs' two tiles the second would be at
// most half full (8 sequences of up to 16384, one without rows, 5 heads to a KV head, 260 / 320 / 380
// rows: 137 / 139 / 155 us in three tiles, 157 / 160 / 171 in two of 256; one of 131072, 300 rows: 223 / 275; 16 of
// up to 500: 50 / 56.  450 rows: 176 in four, 173 in two.  160 / 250 rows: 97 / 105 in two, 108 / 112 in one of
// 256, which these still take).
inline int tree_tile_rows(int64_t flat) { return flat > 256 && flat <= 384 ? 128 : cached_tile_rows(flat); }
inline int64_t fine_floats(int tile_rows, int d) { return tile_rows > kSmallRows ? (int64_t)2 * 128 * d : 0; }
inline int cached_ctas(int tile_rows, int sms) { return tile_rows <= kSmallRows ? sms * kSmallCtasPerSm : sms; }

// Tensor maps: the codes as [n_pages * Hkv, page, d] (V's for the mma.sync
// kernel), the new rows' K and V as [T, Hkv, d] bf16 (for the tcgen05 kernel).
struct CachedMaps {
  CUtensorMap k8, v8, k, v;
};
cudaError_t launch_cached_tc(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches);
cudaError_t launch_tree_tc(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches);
// Longest cache, in tokens, up to which the mma.sync kernel gives each segment
// one CTA, without a list to walk and a merge.  1 / 32 sequences of 8 KV heads (in a
// graph, warm): whole against split 8.0 / 8.9 and 10.1 / 13.3 us at 256 tokens, 14.1 /
// 16.4 and 14.7 / 20.3 at 1000, 21.7 / 27.0 and 20.5 / 27.8 at 2000.
constexpr int kWholeKeys = 1024;
// AttnSplit::extra: what a segment costs beside its units, in units.  The
// mma.sync kernel spends about 6000 cycles to begin and end a segment, 5000 more
// on its own rows' keys and 2300 on a unit: with 1 / 3 / 5, the token batch of
// cached_small.cu took 220 / 207 / 205 us with own keys and 205 / 204 / 206 without,
// blocks of 8 over 16 short sequences 70 / 47 / 42 and 48 / 40 / 41.  The tcgen05
// kernels spend 10 to 20 thousand cycles to end a segment and begin the next, and
// 2000 (split) or 4000 (pairs) on a unit: with 0 / 6, when it was tried, blocks of 32 and 128 took 130 / 106 and 293 /
// 248 us; 4 to 12 are level.
// tree_small.cu spends some 20 thousand cycles on a segment with own rows and 3000 on a unit: with 3 / 5 / 7 / 9 /
// 12, chains of 5 over 32 sequences of up to 32768 tokens took 249 / 236 / 223 / 222 / 222 us, of 8192 107 / 90 / 82 / 82 /
// 82, with d = 64, 4096 tokens 36 / 35 / 36 / 37 / 39, with fp32 outputs, 32768 tokens, 342 / 329 / 328 / 331 / 335.
constexpr int kSmallExtra = 3, kSmallExtraOwn = 5, kTreeExtra = 7, kTcExtra = 6;

cudaError_t launch_cached_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches);
cudaError_t launch_tree_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches);
cudaError_t launch_cached_merge(const CachedParams& p, cudaStream_t st, int* launches);

}  // namespace bdlm
