// kv_cache.cuh -- how the cache's calls and the rotary positions find a token's sequence.
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

// The sequence b with cu[b] <= t < cu[b + 1], by one warp: 32 offsets a step.  -1: none (behind the
// last sequence or before the first); -2: the offsets fall.
__device__ __forceinline__ int find_sequence(const int* cu, int B, int t, int lane) {
  int lo = 0, n = B + 1;  // the last of cu[lo .. lo + n) that is not above t
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && cu[i] <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    if (m == 0u) return -1;
    const int last = 31 - __clz(m);
    n = min(step, n - last * step);
    lo += last * step;
    if (step == 1) break;
  }
  if (lo >= B) return -1;
  return cu[lo] <= t && t < cu[lo + 1] ? lo : -2;
}

}  // namespace fp8gemm
