// kv_cache.cuh -- what the cache's writer and the attention over it share.
#pragma once

#include <cuda_fp16.h>

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

// Two FP8 bytes as an FP16 pair (low byte in the low half): exact for both
// formats.
template <bool kE5M2>
__device__ __forceinline__ uint32_t f8x2_to_f16x2(uint16_t v) {
  uint32_t r;
  if constexpr (kE5M2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(v));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

template <bool kE5M2>
__device__ __forceinline__ float2 f8x2_to_float2(uint16_t v) {
  const uint32_t h = f8x2_to_f16x2<kE5M2>(v);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace fp8gemm
