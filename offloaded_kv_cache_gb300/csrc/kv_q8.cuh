// kv_q8.cuh -- the 8-bit form of a key or value vector: e4m3 codes under one
// power of two (see the header for the format).
#pragma once

#include "kv_internal.cuh"

namespace kvs {

constexpr int kQ8MaxExp = 7;     // 448 * 2^7 = 57344: what f16 still holds
constexpr int kQ8NanScale = 255;
template <class T> __host__ __device__ constexpr int q8_min_exp() { return -110; }
// 2^-9 (the least e4m3 code) * 2^-15 = 2^-24, the least f16
template <> __host__ __device__ constexpr int q8_min_exp<__half>() { return -15; }

// The exponent of a vector whose largest magnitude has the fp32 bits `top`
// (finite): the smallest e with top <= 448 * 2^e = 1.75 * 2^(e + 8), read off
// the bits, so that it is exact.  A subnormal top ends at the lower limit.
__device__ __forceinline__ int q8_exponent(uint32_t top, int least) {
  const int x = (int)(top >> 23) - 127;
  const int e = (top & 0x7FFFFFu) <= 0x600000u ? x - 8 : x - 7;
  return min(max(e, least), kQ8MaxExp);
}
__device__ __forceinline__ float pow2f(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// four codes of x0..x3, x0 in the lowest byte; ties to even, saturating
__device__ __forceinline__ uint32_t q8_codes4(float x0, float x1, float x2, float x3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// the factor of a scale byte; 255 is NaN
__device__ __forceinline__ float q8_scale(uint32_t byte) {
  return byte == (uint32_t)kQ8NanScale ? __uint_as_float(0x7FC00000u)
                                       : __uint_as_float(byte << 23);
}
// four codes -> floats, unscaled
__device__ __forceinline__ void q8_unpack4(uint32_t w, float (&x)[4]) {
  uint32_t a, b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(w & 0xFFFFu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
  const float2 u = __half22float2(*reinterpret_cast<__half2 *>(&a));
  const float2 v = __half22float2(*reinterpret_cast<__half2 *>(&b));
  x[0] = u.x;
  x[1] = u.y;
  x[2] = v.x;
  x[3] = v.y;
}

// 8 floats -> 8 elements of T (16 or 32 bytes), each rounded once
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <class T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(x[0], x[1], T{}), pack2(x[2], x[3], T{}),
                                             pack2(x[4], x[5], T{}), pack2(x[6], x[7], T{}));
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0];
  const float4 b = reinterpret_cast<const float4 *>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <class T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4 *>(p);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(v[i], T{});
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

}  // namespace kvs
