// rope.cuh -- rotary angles and 16-byte vectors of bf16, shared by the kernels
// that rotate queries and keys (the angle's arithmetic is explained in
// rope_write.cu).
#pragma once

#include "common.cuh"

namespace pkv {

// The fraction of a turn that a position advances: frac(f / 2 pi) 2^64, rounded
// down, from the bits of f (a finite double).
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)((bits >> 52) & 2047) - 1023;  // |f| in [2^e, 2^(e + 1))
  const uint64_t m = (bits << 11) | (1ull << 63);   // |f| 2^(63 - e)
  const uint64_t kTwoOverPi = 0xA2F9836E4E441529ull;  // 2 / pi 2^64 = 2^66 / 2 pi
  const uint64_t hi = __umul64hi(m, kTwoOverPi), lo = m * kTwoOverPi;
  // |f| / 2 pi = (hi 2^64 + lo) 2^(e - 129)
  const int s = 65 - e;
  uint64_t r = 0;
  if (s >= 128 || s <= -64)
    r = 0;
  else if (s >= 64)
    r = hi >> (s - 64);
  else if (s > 0)
    r = (hi << (64 - s)) | (lo >> s);
  else
    r = lo << -s;
  return (bits >> 63) ? 0 - r : r;
}

// An infinite or NaN frequency: its pair becomes NaN (a fraction of a turn cannot
// say so).
__device__ __forceinline__ bool no_number(double f) {
  return ((uint64_t)__double_as_longlong(f) >> 52 & 2047) == 2047;
}
constexpr uint32_t kNan = 0x7fffffffu;

// cos and sin of pos turns of `frac` 2^-64 each, times factor.
__device__ __forceinline__ float2 rope_angle(uint64_t frac, uint32_t pos, float factor) {
  const int32_t hi = (int32_t)((frac * pos) >> 32);  // fraction of a turn, as a signed 32-bit one
  float s, c;
  sincospif((float)hi * 4.656612873077393e-10f, &s, &c);  // 2 pi hi / 2^32 = pi hi / 2^31
  return make_float2(c * factor, s * factor);
}

// The same from the nearest quarter turn on: the rest, 30 bits of a turn, loses a
// relative 2^-24 to fp32 (of up to half a turn above). Beside that rounding and the
// function's own the angle is off by the bits of a turn that are left out, less than
// 2^-31 of one, 3e-9 rad: far below an ulp of a value near 1, more than one of a sine or
// cosine below 2^-5. (Keys rounded to 8 bits: of 33.6M, 35 fell to the other side of a
// rounding boundary with the angle above, 24 with this one.)
__device__ __forceinline__ float2 near_angle(uint64_t frac, uint32_t pos, float factor) {
  const uint32_t turn = (uint32_t)((frac * pos) >> 32);
  const uint32_t quarter = (turn + (1u << 29)) >> 30;
  float s, c;
  sincospif((float)(int32_t)(turn - (quarter << 30)) * 4.656612873077393e-10f, &s, &c);
  const bool odd = quarter & 1;
  float cc = odd ? s : c, ss = odd ? c : s;  // a quarter turn on: (c, s) -> (-s, c)
  if ((quarter + 1) & 2) cc = -cc;
  if (quarter & 2) ss = -ss;
  return make_float2(cc * factor, ss * factor);
}

struct Vec8 {
  uint32_t w[4];
};
__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return Vec8{{v.x, v.y, v.z, v.w}};
}
__device__ __forceinline__ void store8(uint16_t* p, const Vec8& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

}  // namespace pkv
