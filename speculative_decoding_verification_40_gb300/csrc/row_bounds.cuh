// Index checks of the row kernels (filtered sampling, top logits, distillation) in debug-bounds builds.  Two of the
// three have no workspace, so that a failed check is recorded in a word of the kernels' own source file, which
// spec_check_status reads beside the workspace's error word; the caller skips the access.  In other builds the checks
// are true and compile away.
#pragma once

#include "common.cuh"

namespace specv {

#ifdef SPEC_DEBUG_BOUNDS
static __device__ uint32_t row_bounds_word;

__device__ __forceinline__ bool index_ok(bool cond) { return bounds_ok(cond, &row_bounds_word); }

// The word, and 0 in its place; for a caller that has waited for the kernels.
static inline cudaError_t take_row_bounds(uint32_t* word) {
  const cudaError_t e = cudaMemcpyFromSymbol(word, row_bounds_word, sizeof(*word));
  if (e != cudaSuccess || *word == 0) return e;
  const uint32_t none = 0;
  return cudaMemcpyToSymbol(row_bounds_word, &none, sizeof(none));
}
#else
__device__ __forceinline__ bool index_ok(bool) { return true; }
#endif

}  // namespace specv
