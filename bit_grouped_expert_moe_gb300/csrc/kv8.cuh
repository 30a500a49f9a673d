// What the kernels of the 8-bit KV cache share (include/kv8.h): the two code
// formats and the checks of the device-side tables.
#pragma once

#include "common.cuh"
#include "kv8.h"

namespace bgmoe {
namespace kv8 {

constexpr float kScaleFloor = 8.673617379884035e-19f;  // 2^-60: the smallest scale of a block not all zero

// Host checks shared by the entry points (kv8_cache.cu).
bool shape_ok(const moe_kv8_shape& s);
bool cache_ok(const moe_kv8_cache* c);
bool aligned(const void* p, uintptr_t n);

// The checks of sequence b's entries in the packed-token table. Every index
// the kernels derive from a table that passes stays inside its array.
__device__ __forceinline__ bool offsets_bad(int lo, int hi, int b, int B, int T) {
  return lo < 0 || hi < lo || hi > T || (b == 0 && lo != 0) || (b == B - 1 && hi != T);
}
__device__ __forceinline__ bool range_bad(int start, int n, int L_max) {
  return start < 0 || n > L_max || start > L_max - n;
}

// The scale that takes magnitudes up to a (finite, >= 0) into the format's
// range. E4M3: a = 1.m * 2^e and 448 = 1.75 * 2^8, so the smallest power of
// two is 2^(e-8), or 2^(e-7) where 1.m > 1.75; an exponent that falls to the
// subnormals or below is lifted by the floor anyway.
template <bool kE4m3>
__device__ __forceinline__ float scale_of(float a) {
  if (!(a > 0.f)) return 0.f;
  if (!kE4m3) return fmaxf(__fdiv_rn(a, 127.f), kScaleFloor);
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return fmaxf(__uint_as_float((uint32_t)max(e, 0) << 23), kScaleFloor);
}

__device__ __forceinline__ float inverse_scale(float s) { return s > 0.f ? __fdiv_rn(1.f, s) : 0.f; }

// Four values (already divided by the scale: |y| <= the format's largest, up
// to the rounding of the reciprocal) as four code bytes, round to nearest even.
template <bool kE4m3>
__device__ __forceinline__ uint32_t encode4(float y0, float y1, float y2, float y3) {
  if (kE4m3) {
    uint16_t lo, hi;  // the first source goes to the upper byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y1), "f"(y0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y3), "f"(y2));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
  // 1.5 * 2^23 + 128 leaves round(y) + 128 in the low byte of the sum
  const float m = 12583040.f;
  const uint32_t a = __float_as_uint(__fadd_rn(y0, m)), b = __float_as_uint(__fadd_rn(y1, m));
  const uint32_t c = __float_as_uint(__fadd_rn(y2, m)), d = __float_as_uint(__fadd_rn(y3, m));
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Byte i (0..3) of a code word as fp32.
template <bool kE4m3>
__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
  if (kE4m3) {
    // sign to bit 15 and exponent, mantissa to bits 13..7 of an fp16: the
    // value times 2^-8 (exponent bias 7 against 15), subnormals included
    const uint32_t odd = (w & 0x80008000u) | ((w >> 1) & 0x3F803F80u);
    const uint32_t w8 = w << 8;
    const uint32_t even = (w8 & 0x80008000u) | ((w8 >> 1) & 0x3F803F80u);
    const float2 o = __half22float2(*reinterpret_cast<const __half2*>(&odd));
    const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&even));
    v[0] = e.x * 256.f;
    v[1] = o.x * 256.f;
    v[2] = e.y * 256.f;
    v[3] = o.y * 256.f;
  } else {
    // 2^23 with the byte as its low mantissa bits is 2^23 + byte
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + i)) - 8388736.f;
  }
}

}  // namespace kv8
}  // namespace bgmoe
