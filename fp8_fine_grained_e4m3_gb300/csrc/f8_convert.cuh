// f8_convert.cuh -- the 1x128 / 128x128 quantisers' per-element arithmetic,
// shared by the quantiser kernels and by the decode GEMM that quantises its
// activations on load: x / s as an IEEE FP32 division (round to nearest),
// then the hardware's round-to-nearest-even, saturating FP8 conversion
// ("news.rkmt.cn/news/5092" section 5.2: s = amax / 448 per block;
// "lpnh.cn/news/2822121" section 6.3: round to nearest).
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"

namespace fp8gemm {

// Two FP32 values -> two FP8 bytes (lo in the low byte), round to nearest
// even, saturate to the format's largest finite value (+-448 e4m3, +-57344
// e5m2).
template <bool kE5M2>
__device__ __forceinline__ uint32_t cvt_f8x2(float lo, float hi) {
  uint16_t r;
  if constexpr (kE5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The format's largest finite value: the divisor of the scale rule.
template <bool kE5M2>
__device__ __forceinline__ float f8_limit() {
  return kE5M2 ? 57344.0f : kE4M3Max;
}

// Four values -> four FP8 bytes (x / s each); kCount: adds to n the
// quotients the conversion clamps (not within +-limit, NaN included).
template <bool kE5M2, bool kCount = false>
__device__ __forceinline__ uint32_t quant4(float4 v, float s, unsigned* n = nullptr) {
  const float q0 = __fdiv_rn(v.x, s), q1 = __fdiv_rn(v.y, s);
  const float q2 = __fdiv_rn(v.z, s), q3 = __fdiv_rn(v.w, s);
  if constexpr (kCount) {
    const float lim = f8_limit<kE5M2>();
    *n += unsigned(!(fabsf(q0) <= lim)) + unsigned(!(fabsf(q1) <= lim)) +
          unsigned(!(fabsf(q2) <= lim)) + unsigned(!(fabsf(q3) <= lim));
  }
  return cvt_f8x2<kE5M2>(q0, q1) | (cvt_f8x2<kE5M2>(q2, q3) << 16);
}

// x / s for many x and one s: Markstein's correction of x times the rounded
// reciprocal ("Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): with r = RN(1/s), q = RN(x r) and the exact remainder
// x - q s, RN(q + (x - q s) r) is the correctly rounded quotient where nothing
// over- or underflows on the way.  `safe` says that for 1x128 quantisation (|x| <= 57344
// s): outside that range of s the plain division is taken.
struct Reciprocal {
  float s, r;
  bool safe;
};
__device__ __forceinline__ Reciprocal reciprocal(float s) {
  return {s, __frcp_rn(s), s >= 1e-25f && s <= 1e25f};
}
__device__ __forceinline__ float quotient(float x, const Reciprocal& d) {
  const float q = __fmul_rn(x, d.r);
  return __fmaf_rn(__fmaf_rn(-q, d.s, x), d.r, q);
}

// quant4 with the scale's reciprocal (d.safe).
template <bool kE5M2>
__device__ __forceinline__ uint32_t quant4(float4 v, const Reciprocal& d) {
  return cvt_f8x2<kE5M2>(quotient(v.x, d), quotient(v.y, d)) |
         (cvt_f8x2<kE5M2>(quotient(v.z, d), quotient(v.w, d)) << 16);
}

// The larger value, or NaN if one is: a NaN in a block must not look like the others' maximum
// (a diverged row would become codes and scales of 0).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// amax / limit: the corrected quotient where that is exact.
template <bool kE5M2>
__device__ __forceinline__ float block_scale(float amax) {
  constexpr float kLimit = kE5M2 ? 57344.f : 448.f;
  const Reciprocal d{kLimit, 1.f / kLimit, true};
  return amax >= 1e-25f && amax <= 1e30f ? quotient(amax, d) : __fdiv_rn(amax, kLimit);
}

// Eight values to codes of one scale; zeros where it is 0 (all zeros, or a maximum so
// small that the scale underflows: the quotient of a 0 there would be NaN).
template <bool kE5M2>
__device__ __forceinline__ uint2 quant8(const float (&v)[8], const Reciprocal& d) {
  const float4 a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
  if (d.safe) return make_uint2(quant4<kE5M2>(a, d), quant4<kE5M2>(b, d));
  if (d.s == 0.f) return make_uint2(0u, 0u);
  return make_uint2(quant4<kE5M2>(a, d.s), quant4<kE5M2>(b, d.s));
}

__device__ __forceinline__ float absmax4(float4 v) {
  return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
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
