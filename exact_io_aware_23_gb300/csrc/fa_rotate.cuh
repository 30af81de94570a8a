// The rotation of pairs by position, as the rotary and the cache-write kernels share it: values loaded
// and stored eight at a time, angles as 64-bit fixed-point turns (fa_rotary.cu says why).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa_paged.cuh"
#include "ptx_sm103.cuh"

namespace fa {
namespace {

constexpr int kUnit = 16;                  // values per unit, 8 pairs

// 8 consecutive values as they lie in memory
template <typename T> struct Raw8 { uint4 w[sizeof(T) / 2]; };
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
}
// ... as fp32, and back (rounded to nearest)
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw8<__half>& r, float (&x)[8]) {
  const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.w[i].x);
    x[4 * i + 1] = __uint_as_float(r.w[i].y);
    x[4 * i + 2] = __uint_as_float(r.w[i].z);
    x[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void pack(const float (&x)[8], Raw8<__nv_bfloat16>& r) {
  r.w[0] = make_uint4(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]), ptx::pack_bf16(x[4], x[5]), ptx::pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void pack(const float (&x)[8], Raw8<__half>& r) {
  r.w[0] = make_uint4(ptx::pack_f16(x[0], x[1]), ptx::pack_f16(x[2], x[3]), ptx::pack_f16(x[4], x[5]), ptx::pack_f16(x[6], x[7]));
}
__device__ __forceinline__ void pack(const float (&x)[8], Raw8<float>& r) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
}

// f / (2 pi) turns as a 64-bit fraction of a turn: the 53-bit significand of f times 2^128/(2 pi),
// shifted by f's exponent, modulo 2^64.  |f| of 2^52 or more, infinities and NaN give 0.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;   // 2^128 / (2 pi)
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)((bits >> 52) & 0x7ff);
  if (e == 0 || e >= 1023 + 52) return 0;
  const uint64_t m = (bits & 0xfffffffffffffull) | (1ull << 52);
  const uint64_t p1 = m * kHi + __umul64hi(m, kLo);
  const uint64_t p2 = __umul64hi(m, kHi) + (p1 < m * kHi ? 1ull : 0ull);
  // f = m * 2^(e - 1075); the fraction is m * 2^128/(2 pi) >> (64 - (e - 1075)), 64 <= shift
  const int s = 64 + 1075 - e - 64;                      // shift of the upper two words, >= 1
  uint64_t r;
  if (s < 64) r = (p1 >> s) | (p2 << (64 - s));
  else r = s < 128 ? p2 >> (s - 64) : 0ull;
  return (bits >> 63) != 0 ? 0ull - r : r;
}

// One thread's unit of every head: where its values lie and its sines and cosines.
struct Unit {
  int lo, hi;               // first value of each group of 8
  bool turns;               // false: values past the rotated part, moved unchanged
};
__device__ __forceinline__ Unit unit_of(int u, const Rotation& r) {
  Unit t;
  t.turns = u < r.rot / kUnit;
  const bool halves = t.turns && !r.interleaved;
  t.lo = halves ? 8 * u : kUnit * u;
  t.hi = halves ? r.rot / 2 + 8 * u : kUnit * u + 8;
  return t;
}
__device__ __forceinline__ void angles(const uint64_t (&frac)[8], int pos, const Rotation& r,
                                       float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t w = (uint64_t)(int64_t)pos * frac[i];
    // the upper 32 bits, signed: half turns in [-1, 1)
    const float half_turns = (float)(int32_t)(uint32_t)(w >> 32) * 4.656612873077393e-10f;
    float sn, cs;
    sincospif(half_turns, &sn, &cs);
    c[i] = cs * r.mscale;
    s[i] = sn * r.mscale * r.sign;
  }
}
// (a, b) of the unit's 8 pairs turned in place; the pairs are (x[i], y[i]) or neighbours
__device__ __forceinline__ void turn8(float (&x)[8], float (&y)[8], bool interleaved,
                                      const float (&c)[8], const float (&s)[8]) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1], p = y[2 * i], q = y[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = a * s[i] + b * c[i];
      y[2 * i] = p * c[i + 4] - q * s[i + 4];
      y[2 * i + 1] = p * s[i + 4] + q * c[i + 4];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = y[i];
      x[i] = a * c[i] - b * s[i];
      y[i] = a * s[i] + b * c[i];
    }
  }
}

template <typename T>
__device__ __forceinline__ void turn_raw(Raw8<T>& lo, Raw8<T>& hi, bool interleaved, const float (&c)[8],
                                         const float (&s)[8]) {
  float x[8], y[8];
  unpack(lo, x);
  unpack(hi, y);
  turn8(x, y, interleaved, c, s);
  pack(x, lo);
  pack(y, hi);
}

}  // namespace
}  // namespace fa
