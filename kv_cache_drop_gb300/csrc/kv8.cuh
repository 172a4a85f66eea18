// A cache row in 8 bits, shared by the kernels that write it, read it back
// (kv8.cu) and attend over it (decode8.cu).
//
// A head row of 64 is 64 e4m3 values and one power of two 2^s, kept as the
// byte s + 127 (e8m0).  s is the smallest in -127 .. 127 with
// max |x| <= 448 * 2^s over the row's finite x; a code is x * 2^-s rounded to
// the nearest e4m3 value, ties to even, and NaN where x is not finite.  e4m3 is
// a floating format: a scale that is no power of two would gain the row's one
// largest value at most half a step, and cost four bytes instead of one and a
// rounding in every product.
#pragma once

#include "common.cuh"

#include <algorithm>
#include <cmath>

namespace akv {

// |x| as bits, 0 where x is not finite: ordered as |x| is
__device__ __forceinline__ uint32_t kv8_size(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// scale byte of a row whose largest kv8_size is `top`: 448 = 1.75 * 2^8
__device__ __forceinline__ uint32_t kv8_scale(uint32_t top) {
  const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
  return (uint32_t)max(0, e);
}
// 2^-s: its exponent is 254 - (s + 127), from 7 to 254
__device__ __forceinline__ float kv8_inverse(uint32_t scale) {
  return __uint_as_float((254u - scale) << 23);
}
// 2^s; 2^-127 is no normal fp32 number
__device__ __forceinline__ float kv8_power(uint32_t scale) {
  return __uint_as_float(scale ? scale << 23 : 0x400000u);
}

// Codes of four values, the first in the lowest byte.  The conversion turns an
// infinity into 448; 0 * x makes it NaN first.
__device__ __forceinline__ uint32_t kv8_codes(const float *x, float inverse) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fmaf(x[e], 0.f, x[e] * inverse);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// Two codes as an fp16 pair (exact), the lower byte in the lower half
__device__ __forceinline__ uint32_t kv8_pair(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}
// four codes times `power`
__device__ __forceinline__ void kv8_floats(uint32_t codes, float power, float *x) {
  const uint32_t a = kv8_pair((uint16_t)codes), b = kv8_pair((uint16_t)(codes >> 16));
  const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&a));
  const float2 w = __half22float2(*reinterpret_cast<const __half2 *>(&b));
  x[0] = u.x * power;
  x[1] = u.y * power;
  x[2] = w.x * power;
  x[3] = w.y * power;
}

// Frequencies in turns: theta / 2 pi = hi 2^-32 + lo 2^-64 for the double theta, so
// that a position times it modulo 1 is off by less than 1.3 * 2^-32 turns (the floor, and a
// quarter for lo's rounding), in two integer products, for any position.
struct Turns {
  int32_t hi[kD / 2], lo[kD / 2];
};
__device__ __forceinline__ uint32_t turn_of(int hi, int lo, int pos) {
  return (uint32_t)pos * (uint32_t)hi + (uint32_t)__mulhi(pos, lo);
}

// cos and sin: the angle is good to 2^-24 of itself and 1.9e-9 (theta's own rounding,
// 2^-53 of it, is beside that 2.4e-7 where the angle is 2^31)
__device__ __forceinline__ void turn_cs(int hi, int lo, int pos, float *c, float *s) {
  sincospif((float)(int)turn_of(hi, lo, pos) * 4.656612873e-10f, s, c);
}
inline Turns turns_of(const RopeTheta &th) {
  // 2^32 / 2 pi in two doubles: one would leave 23 bits of lo where theta is 1, and the
  // turn off by 90 of 2^-32 at position 2^31
  const double c0 = 0x1.45f306dc9c883p-3 * 4294967296.0, c1 = -0x1.6b01ec5417056p-57 * 4294967296.0;
  Turns turns;
  for (int f = 0; f < kD / 2; ++f) {
    const double t = th.th[f] * c0, rest = std::fma(th.th[f], c1, std::fma(th.th[f], c0, -t));
    const double hi = std::rint(t), lo = std::rint(((t - hi) + rest) * 4294967296.0);
    turns.hi[f] = (int32_t)(uint32_t)(int64_t)hi;
    turns.lo[f] = (int32_t)std::min(std::max(lo, -2147483648.0), 2147483647.0);
  }
  return turns;
}

}  // namespace akv
