// vec.cuh -- eight consecutive activations (BF16 or FP32) at a time, as FP32.
#pragma once

#include "common.cuh"

namespace fp8gemm {

template <class T>
struct Raw8;  // eight elements as they lie in memory
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Raw8<float> {
  uint4 a, b;
};

__device__ __forceinline__ Raw8<__nv_bfloat16> load8(const __nv_bfloat16* p) {
  return {*reinterpret_cast<const uint4*>(p)};
}
__device__ __forceinline__ Raw8<float> load8(const float* p) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  return {q[0], q[1]};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Raw8<__nv_bfloat16>& r) {
  *reinterpret_cast<uint4*>(p) = r.a;
}
__device__ __forceinline__ void store8(float* p, const Raw8<float>& r) {
  uint4* q = reinterpret_cast<uint4*>(p);
  q[0] = r.a;
  q[1] = r.b;
}

__device__ __forceinline__ void zero8(Raw8<__nv_bfloat16>& r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero8(Raw8<float>& r) {
  r.a = make_uint4(0, 0, 0, 0);
  r.b = make_uint4(0, 0, 0, 0);
}

// A BF16 is the upper half of the FP32 of the same value.
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Rounded to nearest even where the type has fewer bits.
__device__ __forceinline__ void pack8(const float (&v)[8], Raw8<__nv_bfloat16>& r) {
  r.a = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                   bf16x2_bits(v[6], v[7]));
}
__device__ __forceinline__ void pack8(const float (&v)[8], Raw8<float>& r) {
  r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                   __float_as_uint(v[3]));
  r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                   __float_as_uint(v[7]));
}

// Sums rounded to the type.  For BF16 the instruction rounds the exact sum once;
// that is also the FP32 sum rounded to BF16, for the FP32 sum is exact unless one
// operand is 2^-16 of the other or less, and then both are the larger one.
__device__ __forceinline__ Raw8<__nv_bfloat16> add8(const Raw8<__nv_bfloat16>& x,
                                                    const Raw8<__nv_bfloat16>& y) {
  const uint32_t a[4] = {x.a.x, x.a.y, x.a.z, x.a.w}, b[4] = {y.a.x, y.a.y, y.a.z, y.a.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a[i]),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b[i]));
    c[i] = *reinterpret_cast<const uint32_t*>(&s);
  }
  return {make_uint4(c[0], c[1], c[2], c[3])};
}
__device__ __forceinline__ Raw8<float> add8(const Raw8<float>& x, const Raw8<float>& y) {
  float a[8], b[8];
  unpack8(x, a);
  unpack8(y, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] += b[i];
  Raw8<float> r;
  pack8(a, r);
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace fp8gemm
