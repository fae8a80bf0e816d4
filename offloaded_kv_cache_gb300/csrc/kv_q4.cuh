// kv_q4.cuh -- the 4-bit form of a key or value vector: integers c of 4 bits, an e4m3
// scale s for every 16 channels, one power of two (see the header for the format).
#pragma once

#include <type_traits>

#include "kv_internal.cuh"
#include "kv_q8.cuh"

namespace kvs {

constexpr int kQ4Group = 16;                    // channels of a scale
constexpr int kQ4Scales = kHeadDim / kQ4Group;  // bytes of scales a vector
constexpr int kQ4Bytes = kHeadDim / 2;          // bytes of codes a vector
constexpr int kQ4MaxExp = 4;                    // 7 * 448 * 2^4 = 50176: what f16 still holds
constexpr int kQ4NanPower = 255;
// (the least exponents are the 8-bit form's: 1 * 2^-9 * 2^-15 = 2^-24, the least f16)

// The exponent of a vector whose largest magnitude has the fp32 bits `top` (finite): the
// smallest e with top <= 3136 * 2^e = 1.53125 * 2^(e + 11).
__device__ __forceinline__ int q4_exponent(uint32_t top, int least) {
  const int x = (int)(top >> 23) - 127;
  const int e = (top & 0x7FFFFFu) <= 0x440000u ? x - 11 : x - 10;
  return min(max(e, least), kQ4MaxExp);
}
// two e4m3 codes -> floats
__device__ __forceinline__ float2 e4m3_pair(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<__half2 *>(&h));
}
// The code of the smallest s with 7 s >= top, 448 at most.  The code nearest to top / 7 is
// that one or the one below (a quotient that rounds onto a code is one with it or above),
// and 7 s is exact.
__device__ __forceinline__ uint32_t q4_scale_code(float top, float &s) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(top * (1.f / 7.f)));
  uint32_t code = c & 0xFFu;
  s = e4m3_pair(code).x;
  if (7.f * s < top && code < 0x7Eu) s = e4m3_pair(++code).x;
  return code;
}
// within 2^-23 of 1 / x
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Eight channels as nibbles c + 8, x0 in the lowest; top: the largest magnitude of the scale's
// channels times 2^-e.  t = x / (s 2^e) + 1/2 + 8 + 2^-15 + 2^7 has its integer part, less 2^7,
// in its third byte alone.  The quotient by an approximate reciprocal is off by 2^-19 at most,
// and t is rounded to 2^-16: a tie stays at or above it, and 16-bit data, which differ from a tie
// (8 significant bits) by 2^-11 of it at least, 2^-12 here, stay below.  fp32 data may differ by
// less: a fraction of 4 * 2^-16 or more shows that no border is near; else the integer found is
// compared with its two borders, which are exact.  (All lanes call.)
template <class T>
__device__ __forceinline__ uint32_t q4_codes8(const float (&x)[8], float top, float s, int e, T) {
  const float down = pow2f(-e), f = s == 0.f ? 0.f : rcp(s) * down;
  float t[8];
  uint32_t fraction = 0xFFFFu;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(x[i], f, 136.5f + 0x1p-15f);
    fraction = min(fraction, __float_as_uint(t[i]) & 0xFFFFu);
  }
  if (sizeof(T) == 4 && fraction < 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = __uint_as_float(__float_as_uint(t[i]) & ~0xFFFFu) - 136.f;  // floor(t), less
      const float y = x[i] * down, border = fmaf(c, s, -0.5f * s);
      if (border > y) t[i] -= 1.f;
      if (border + s <= y && s != 0.f) t[i] += 1.f;
    }
  }
  if (__any_sync(0xFFFFFFFFu, 7.f * s < top)) {  // (a power at its limit)
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = fminf(fmaxf(t[i], 129.5f), 143.5f);
  }
  // the third bytes, four even and four odd ones side by side
  uint32_t half[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    half[i] = __byte_perm(__byte_perm(__float_as_uint(t[i]), __float_as_uint(t[i + 2]), 0x0062),
                          __byte_perm(__float_as_uint(t[i + 4]), __float_as_uint(t[i + 6]), 0x0062), 0x5410);
  return half[1] * 16u + half[0];
}
// The factor of a vector's power byte; 255 is NaN.
__device__ __forceinline__ float q4_power(uint32_t byte) { return q8_scale(byte); }
// (Integers put into the mantissa of a float of known exponent: a published method, for 4 bits
// and f16 in Kim, Henry, Fahim and Hassan Awadalla, "Who Says Elephants Can't Run: Bringing
// Large Scale MoE Models into Cloud Scale Production", 2022.)
// n = c + 8 (below 16) times f = s 2^e: n is put into the mantissa of 2^23 + n (f16: 1024 + n,
// bf16: 128 + n, two at a time); what is taken off again leaves c, and c f is exact in every
// type.
__device__ __forceinline__ float q4_value(uint32_t n, float f) {
  return (__uint_as_float(n | 0x4B000000u) - 8388616.f) * f;
}
// four nibbles -> four floats
__device__ __forceinline__ float4 q4_values4(uint32_t w, float f) {
  return make_float4(q4_value(w & 15u, f), q4_value((w >> 4) & 15u, f), q4_value((w >> 8) & 15u, f),
                     q4_value((w >> 12) & 15u, f));
}
// The mask of nibbles 0 and 4 of a word, and the exponent of two 16-bit elements, in registers:
// so that one operation takes both (of two immediates the compiler makes two).
template <class T> struct Q4Bits {
  uint32_t mask, one;
  __device__ __forceinline__ Q4Bits() {
    constexpr bool f16 = std::is_same<T, __half>::value;
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(mask));
    asm volatile("mov.b32 %0, %1;" : "=r"(one) : "n"(f16 ? 0x64006400 : 0x43004300));
  }
  // c f of nibbles 0 and 4.  bf16: (128 + n) f - 136 f in one fma, g = -136 f: f has 4
  // significant bits and 17 * 15 has 8, so that g is exact.  (f16: 1032 f would be past its range.)
  __device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t f, [[maybe_unused]] uint32_t g) const {
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "r"(mask), "r"(one));
    if constexpr (std::is_same<T, __half>::value) {
      asm("add.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(0xE408E408u));
      asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(f));
    } else {
      asm("fma.rn.bf16x2 %0, %0, %1, %2;" : "+r"(x) : "r"(f), "r"(g));
    }
    return x;
  }
  // eight nibbles times the factor in both halves of f, in order
  __device__ __forceinline__ uint4 expand(uint32_t w, uint32_t f) const {
    uint32_t g = 0;
    if constexpr (!std::is_same<T, __half>::value)
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(g) : "r"(f), "r"(0xC308C308u));
    const uint32_t x0 = pair(w, f, g), x1 = pair(w >> 4, f, g), x2 = pair(w >> 8, f, g),
                   x3 = pair(w >> 12, f, g);
    return make_uint4(__byte_perm(x0, x1, 0x5410), __byte_perm(x2, x3, 0x5410),
                      __byte_perm(x0, x1, 0x7632), __byte_perm(x2, x3, 0x7632));
  }
};
template <> struct Q4Bits<float> {};
// eight nibbles, stored as eight elements
__device__ __forceinline__ void q4_store8(float *p, uint32_t w, float f, const Q4Bits<float> &) {
  reinterpret_cast<float4 *>(p)[0] = q4_values4(w, f);
  reinterpret_cast<float4 *>(p)[1] = q4_values4(w >> 16, f);
}
template <class T>
__device__ __forceinline__ void q4_store8(T *p, uint32_t w, float f, const Q4Bits<T> &bits) {
  *reinterpret_cast<uint4 *>(p) = bits.expand(w, pack2(f, f, T{}));
}

}  // namespace kvs
