// Rows of the 8-bit pool (sm_103a): e4m3 codes under one power-of-two scale.
//
// A row is the K (or V) of one token and kv head. With a = its largest
// magnitude, its exponent is the least e >= kLeastExp with a <= 448 * 2^e, its
// codes are the e4m3 numbers nearest to x * 2^-e (ties to even), and its scale
// byte is e + 127: value = code * 2^(scale - 127). e4m3 is a floating format, so
// a scale of 448 / a exactly would gain no accuracy over the next power of two;
// the power makes the division exact, and code * 2^e, four significant bits, is
// exactly a bf16: rows read back are exact, and attention over rows turned into
// bf16 is attention over what the pool holds. (Under 2^120, the scale of rows above
// 1.75 * 2^127, a code is 240 at most: 256 * 2^120 is no bf16, nor an fp32.) A row with an infinity or a NaN
// is held as NaN: codes 0 and scale 255, 0 times fp32's 2^128, an infinity. (So no
// code is a NaN, and a weight of 0 leaves nothing of a masked row.)
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace pkv {

// 2^-117 times the smallest code, 2^-9, is bf16's (and fp32's) smallest normal number.
constexpr int kLeastExp = -117;
constexpr uint32_t kNanScale = 255u;
constexpr uint32_t kTopScale = 247u;  // 2^120

// Scale byte of a row whose largest bf16 magnitude has the bits `amax`
// (exponent E, mantissa M): 448 = 1.75 * 2^8, so e is E - 127 - 8, plus one where
// 1.M is above 1.75 (M above 0x60). The sum carries into the exponent just there.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int s = static_cast<int>((amax + 0x1fu) >> 7) - 8;
  return amax >= 0x7f80u ? kNanScale : static_cast<uint32_t>(max(s, kLeastExp + 127));
}

// 2^(scale - 127), NaN for kNanScale. (Bytes below 10 stand in no pool that was
// written by this library: 0 counts as 0.)
__device__ __forceinline__ float scale_value(uint32_t s) {
  const float f = __uint_as_float(s << 23);
  return fmaf(f, 0.f, f);  // an infinity times 0 is a NaN
}

// scale - 127 as a float, NaN for kNanScale.
__device__ __forceinline__ float scale_exponent(uint32_t s) {
  const float e = __uint_as_float(0x4b000000u | s) - 8388735.f;  // (2^23 + s) - (2^23 + 127)
  return fmaf(__uint_as_float(s << 23), 0.f, e);
}

// Two floats to two e4m3 codes (a in the low byte), to nearest even; values
// above 448 become 448.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Two e4m3 codes (low 16 bits) to two floats.
__device__ __forceinline__ float2 e4m3_float2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Largest of the magnitudes' bits of eight bf16.
__device__ __forceinline__ uint32_t amax8(const uint4& v) {
  auto max2 = [](uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  };
  const uint32_t k = 0x7fff7fffu;
  const uint32_t m = max2(max2(v.x & k, v.y & k), max2(v.z & k, v.w & k));
  return max(m & 0xffffu, m >> 16);
}

// x * m with subnormal numbers kept, which the build flushes elsewhere.
__device__ __forceinline__ float mul_subnormal(float x, float m) {
  float r;
  asm("mul.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(m));
  return r;
}

// Four codes of 256 (0x78) at most: those of 256 become 240, the code before it.
__device__ __forceinline__ uint32_t below_256(uint32_t c) {
  return c - ((c & (c >> 1) & (c >> 2) & (c >> 3) & 0x08080808u) >> 3);  // bits 3 .. 6 are set
}

// Eight bf16 to eight codes under a scale byte below kTopScale.
__device__ __forceinline__ uint2 quant8_usual(const uint4& v, uint32_t s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float m = __uint_as_float((254u - s) << 23);  // 2^(127 - s)
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x2(mul_subnormal(bf16_lo(w[i]), m), mul_subnormal(bf16_hi(w[i]), m));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The same under any scale byte. (What is rare comes last: a branch ahead of the
// conversions took 2% of a write of 16001 rows and 4% of one of 64.)
__device__ __forceinline__ uint2 quant8(const uint4& v, uint32_t s) {
  uint2 r = quant8_usual(v, s);
  if (s >= kTopScale)
    r = s == kNanScale ? make_uint2(0u, 0u) : make_uint2(below_256(r.x), below_256(r.y));
  return r;
}

// Four codes times m, as four bf16.
__device__ __forceinline__ uint2 dequant4(uint32_t codes, float m) {
  const float2 a = e4m3_float2(codes & 0xffffu), b = e4m3_float2(codes >> 16);
  return make_uint2(pack_bf16x2(a.x * m, a.y * m), pack_bf16x2(b.x * m, b.y * m));
}

}  // namespace pkv
