// kv_q8.cuh -- the 8-bit form of a key or value vector: e4m3 codes under one
// power of two (see the header for the format).
#pragma once

#include "kv_internal.cuh"

namespace kvs {

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31: with 2^shift >= d > 2^(shift-1) and mul =
// floor(2^32 (2^shift - d) / d) + 1, 2^32 + mul is 2^(32+shift) / d + e, 0 < e <= 1, so n
// (2^32 + mul) / 2^(32+shift) exceeds n / d by less than 2^-(shift+1) < 1 / d, and its
// floor is that of n / d.  (A division by a variable takes four times as long.)
struct Divisor {
  uint32_t mul;
  int shift;
  static Divisor of(int d) {
    int s = 0;
    while ((1ll << s) < d) ++s;
    return Divisor{(uint32_t)((((1ull << s) - d) << 32) / d + 1), s};
  }
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
  }
};

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
// 8 elements -> floats
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
// The largest magnitude among 8 elements, as bits: they order as the values do,
// infinities and NaN above all.
__device__ __forceinline__ uint32_t q8_top(const uint4 (&w)[1]) {  // two 16-bit elements a word
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vmaxu2(__vmaxu2(w[0].x & m, w[0].y & m), __vmaxu2(w[0].z & m, w[0].w & m));
  return max(t & 0xFFFFu, t >> 16);
}
__device__ __forceinline__ uint32_t q8_top(const uint4 (&w)[2]) {
  const uint32_t m = 0x7FFFFFFFu;
  return max(max(max(w[0].x & m, w[0].y & m), max(w[0].z & m, w[0].w & m)),
             max(max(w[1].x & m, w[1].y & m), max(w[1].z & m, w[1].w & m)));
}
// such bits as those of an fp32 number
__device__ __forceinline__ uint32_t q8_top_f32(uint32_t t, float) { return t; }
__device__ __forceinline__ uint32_t q8_top_f32(uint32_t t, __nv_bfloat16) { return t << 16; }
__device__ __forceinline__ uint32_t q8_top_f32(uint32_t t, __half) {
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)t)));
}
// Eight elements times 2^-e as codes.  f16 scales in f16: exact, but for results
// below 2^-14, which round to a code of 0 as they would without that.
__device__ __forceinline__ uint2 q8_codes8(const uint4 (&w)[1], int e, __half) {
  const uint32_t f = (uint32_t)(15 - e) << 10, f2 = f | (f << 16);
  const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
  uint16_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(v[i]), "r"(f2));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c[i]) : "r"(y));
  }
  return make_uint2((uint32_t)c[0] | ((uint32_t)c[1] << 16), (uint32_t)c[2] | ((uint32_t)c[3] << 16));
}
template <class T, int N>
__device__ __forceinline__ uint2 q8_codes8(const uint4 (&w)[N], int e, T) {
  float x[8];
  load8(reinterpret_cast<const T *>(&w), x);
  const float s = pow2f(-e);
  return make_uint2(q8_codes4(x[0] * s, x[1] * s, x[2] * s, x[3] * s),
                    q8_codes4(x[4] * s, x[5] * s, x[6] * s, x[7] * s));
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
}  // namespace kvs
