// kv_cache.cuh -- what the cache's writer and the attention over it share.
#pragma once

#include "common.cuh"

namespace fp8gemm {

// Tokens [t0, t0 + n) of the packed token axis belong to sequence b: by the
// B + 1 offsets cu, or, without them, T / B to each.  False where the offsets
// leave [0, T], fall, or give a sequence more than most.
__device__ __forceinline__ bool sequence_tokens(const int* cu, int b, int B, int T, int most,
                                                int* t0, int* n) {
  if (cu == nullptr) {
    *n = T / B;
    *t0 = b * *n;
    return true;
  }
  const int lo = cu[b], hi = cu[b + 1];
  *t0 = lo;
  *n = hi - lo;
  return lo >= 0 && hi >= lo && hi <= T && hi - lo <= most;
}

}  // namespace fp8gemm
