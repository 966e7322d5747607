// abi_internal.h -- what the C entry points in other files share with abi.cu:
// errors, device checks, the tensor-map encoder, launch counting and timing.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/bdlm_attn.h"

namespace bdlm {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Records the message of a failing status and returns it.
bdlm_status abi_fail(bdlm_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// SM count of the current device; an error status when it is not sm_103.
bdlm_status abi_device(int* sms);
bdlm_status abi_encoder(EncodeTiledFn* fn);
uint64_t abi_wait_limit_ns();

enum AbiTimer { ABI_T_APPEND, ABI_T_ATTN_CACHED, ABI_T_CACHED_MERGE, ABI_T_WEIGHTS, ABI_T_EVICT,
                ABI_T_TREE_MASK, ABI_T_VERIFY, ABI_T_COMMIT };
// Brackets a launch for bdlm_timing_report (nothing when timing is off).
void* abi_timer_begin(AbiTimer kind, cudaStream_t st);
void abi_timer_end(void* timer);
// Counts launches and turns a launch error into a status.
bdlm_status abi_finish(cudaError_t e, int launches, const char* what);

}  // namespace bdlm
