// Codes of 8-bit pages and of key bounds: conversions and the scales they go with.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fa_internal.cuh"

namespace fa {

// The element of a page that holds values of type T.
template <typename T, int kStore>
struct StoredAs { using type = std::conditional_t<kStore == FA_PAGES_16BIT, T, uint8_t>; };

// The smallest power of two, at least 2^-100, whose `largest` (127 for int8, 448 for e4m3) reaches the
// finite value with these bits: 127 = 2^6 * 1.984375, 448 = 2^8 * 1.75.
template <bool kInt8>
__device__ __forceinline__ float power_scale(uint32_t bits) {
  constexpr uint32_t kTop = kInt8 ? 0x7e0000u : 0x600000u;     // the largest code's fraction
  constexpr int kExp = kInt8 ? 6 : 8;
  const int e = (int)(bits >> 23) - kExp + ((bits & 0x7fffffu) > kTop ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 27) << 23);          // 27: 2^-100
}

// four values to bytes, the first one lowest; saturated
__device__ __forceinline__ uint32_t pack_s8(int a, int b, int c, int d) {
  uint32_t hi, r;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(hi) : "r"(d), "r"(c), "r"(0));
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(b), "r"(a), "r"(hi));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{ .reg .b16 x, y; cvt.rn.satfinite.e4m3x2.f32 x, %2, %1; cvt.rn.satfinite.e4m3x2.f32 y, %4, %3; mov.b32 %0, {x, y}; }"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ void unpack_e4m3(uint32_t c, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{ .reg .b16 x, y; mov.b32 {x, y}, %2; cvt.rn.f16x2.e4m3x2 %0, x; cvt.rn.f16x2.e4m3x2 %1, y; }"
      : "=r"(lo), "=r"(hi) : "r"(c));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// Four codes of a register (bytes 0 to 3) as two pairs of fp16: bytes 0, 1 and 2, 3, or 0, 2 and 1, 3.
// int8: the byte with its sign turned becomes the low bits of 1024 + x + 128, from which 1152 is taken.
template <bool kInt8, bool kApart>
__device__ __forceinline__ void codes(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (kInt8) {
    x ^= 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));            // 1152
    auto pair = [&](uint32_t sel) {
      const uint32_t y = __byte_perm(x, 0x64646464u, sel);
      const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&y), bias);
      return *reinterpret_cast<const uint32_t*>(&h);
    };
    lo = pair(kApart ? 0x4240 : 0x4140);
    hi = pair(kApart ? 0x4341 : 0x4342);
  } else {
    if constexpr (kApart) x = __byte_perm(x, 0u, 0x3120);
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
        : "=r"(lo), "=r"(hi) : "r"(x));
  }
}

}  // namespace fa
