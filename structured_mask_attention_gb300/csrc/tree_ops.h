// tree_ops.h -- parameters and launchers of the calls on drafted trees that need no
// attention: what the rows see, and which drafts the target accepts.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"

namespace bdlm {

// Rows of a tree: its parents and what the walk needs of every row are held in
// shared memory (24 bytes each).
constexpr int kMaxTreeRows = 4096;

struct TreeMaskParams {
  CacheDesc c;
  RowsDesc r;
  const int32_t* parents;  // [T]
  uint32_t* vis;           // [T, words]
  int words;
  int32_t* positions;      // [T]
  uint32_t* status;
};
cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t st, int* launches);

struct VerifyParams {
  RowsDesc r;
  int n_seqs;
  const int32_t *parents, *tokens;  // [T]
  const void *target, *draft;       // [T, V], rows a stride of elements apart; draft may be null
  int bf16;
  int64_t V, target_stride, draft_stride;
  const float *uniforms, *sample;   // [T], [n_seqs]
  int32_t* path;                    // [n_seqs, max_path]
  int max_path;
  int32_t *accepted, *next_token;   // [n_seqs]
  uint32_t* status;
};
cudaError_t launch_tree_verify(const VerifyParams& p, int sms, cudaStream_t st, int* launches);

}  // namespace bdlm
