// Scores that are capped by a tanh and lowered by a bias linear in distance (fa_score_mod): the
// arithmetic that the forward, both passes of the backward and the paged kernel share.
//
//     y = cap * tanh(u / cap) - slope |i - j|,  u = scale * (q . k);   dy/du = 1 - tanh^2(u / cap)
//
// All in the log2 domain, as the softmax is.  The tanh is what costs: through the exponential,
// 1 - 2 / (1 + exp 2x), it takes two more special-function operations a score beside the softmax's
// one, and that unit (16 a clock on an SM) then sets the pace of the whole attention at a third of
// its speed.  Scores far below the cap are the common case, so where no score of a warp's tile
// exceeds the cap, tanh(x) = x P(x^2) on |x| <= 1 with P of degree 6 (minimax for the relative
// error, found by exchange: 5.0e-8, less than fp32's own rounding), eight packed operations for two
// scores on the multiply-add pipe; else the exponential form, for the whole tile.
#pragma once

#include <cuda_runtime.h>
#include <math.h>

#include "fa_internal.cuh"
#include "ptx_sm103.cuh"

namespace fa {

// P's coefficients, ascending
constexpr double kTanhPoly[7] = {0.9999999502407381,   -0.3333283915308157,  0.13325204075948163,
                                 -0.05345702957318134, 0.02028998043217086,  -0.0062033791124837,
                                 0.0010410226362182575};

// Fills the kernels' form of the score arguments for raw products q . k; false when the cap is out
// of the range fp32 can hold them in.
inline bool make_score(const fa_score_mod* m, float scale, ScoreArgs* out) {
  *out = ScoreArgs{};
  if (m == nullptr) return true;
  out->slopes = m->alibi_slopes;
  out->prefix = m->prefix_lens;
  if (m->softcap > 0.f) {
    const double r = (double)scale / (double)m->softcap;
    out->cap_log2 = (float)((double)m->softcap * 1.4426950408889634);
    out->c_exp = (float)(2.0 * r * 1.4426950408889634);
    if (!isfinite(out->cap_log2) || !isfinite(out->c_exp) || !(out->cap_log2 > 0.f)) return false;
    out->poly_limit = (float)(1.0 / r);
    double p = r;
    for (int i = 0; i < 7; ++i, p *= r * r) {
      out->poly[i] = (float)(kTanhPoly[i] * p);
      if (!isfinite(out->poly[i])) out->poly_limit = -1.f;      // a tiny cap: always the exponential
    }
    if (!isfinite(out->poly_limit)) out->poly_limit = 3.4e38f;
  }
  return true;
}

// tanh(scale s / cap) of two raw products, |scale s| <= cap
__device__ __forceinline__ float2 tanh_poly(float2 s, const ScoreArgs& k) {
  const float2 z = ptx::mul2(s, s);
  float2 p = make_float2(k.poly[6], k.poly[6]);
#pragma unroll
  for (int i = 5; i >= 0; --i) p = ptx::fma2(p, z, make_float2(k.poly[i], k.poly[i]));
  return ptx::mul2(p, s);
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// the same for any s: 1 - 2 / (1 + exp 2x); the exponential may overflow to infinity
__device__ __forceinline__ float2 tanh_exp(float2 s, const ScoreArgs& k) {
  const float r0 = rcp(1.f + ptx::ex2(s.x * k.c_exp)), r1 = rcp(1.f + ptx::ex2(s.y * k.c_exp));
  return make_float2(fmaf(-2.f, r0, 1.f), fmaf(-2.f, r1, 1.f));
}
// one score by the better form for it
__device__ __forceinline__ float tanh_one(float s, const ScoreArgs& k) {
  const float2 p = tanh_poly(make_float2(s, s), k);
  return fabsf(s) <= k.poly_limit ? p.x : fmaf(-2.f, rcp(1.f + ptx::ex2(s * k.c_exp)), 1.f);
}

// Whether a tile of scores s[0..n) may take the polynomial (the same answer in the whole warp).
template <int N>
__device__ __forceinline__ bool poly_fits(const float (&s)[N], float limit) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < N; e += 2) m[(e >> 1) & 3] = ptx::max3(m[(e >> 1) & 3], fabsf(s[e]), fabsf(s[e + 1]));
  const float mx = ptx::max3(ptx::max3(m[0], m[1], m[2]), m[3], m[3]);
  return __all_sync(0xffffffffu, mx <= limit);
}

// The forms of one tile's scores: which tanh, and whether there is a bias.
enum : int { kCapNone = 0, kCapPoly = 1, kCapExp = 2 };
template <int kCap>
__device__ __forceinline__ float2 tanh_of(float2 s, const ScoreArgs& k) {
  if constexpr (kCap == kCapPoly) return tanh_poly(s, k);
  else return tanh_exp(s, k);
}
// -slope |i - j| for score e of a row (or column) whose distances run on by one from `first`:
// base = slope * first, step = slope
__device__ __forceinline__ float biased(float x, float base, float step, int e) {
  return x - fabsf(fmaf(step, (float)e, base));
}

// Calls body(cap form, with or without bias) as compile-time constants, the same one in the warp.
template <int V> struct Const { static constexpr int value = V; };
template <int N, typename Body>
__device__ __forceinline__ void with_score(const float (&s)[N], const ScoreArgs& k, Body&& body) {
  const bool bias = k.slopes != nullptr;
  if (k.cap_log2 == 0.f) {
    if (bias) body(Const<kCapNone>(), Const<1>());
    else body(Const<kCapNone>(), Const<0>());
  } else if (poly_fits(s, k.poly_limit)) {
    if (bias) body(Const<kCapPoly>(), Const<1>());
    else body(Const<kCapPoly>(), Const<0>());
  } else {
    if (bias) body(Const<kCapExp>(), Const<1>());
    else body(Const<kCapExp>(), Const<0>());
  }
}

// Scores s[0..N) of one row turned into the log2 domain in place.
template <int N>
__device__ __forceinline__ void score_row(float (&s)[N], const ScoreArgs& k, float c, float base, float step) {
  with_score(s, k, [&](auto cap, auto bias) {
    constexpr int kCap = decltype(cap)::value;
    const float2 m2 = kCap == kCapNone ? make_float2(c, c) : make_float2(k.cap_log2, k.cap_log2);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      float2 x = make_float2(s[e], s[e + 1]);
      if constexpr (kCap != kCapNone) x = tanh_of<kCap>(x, k);
      x = ptx::mul2(x, m2);
      if constexpr (decltype(bias)::value != 0) {
        x.x = biased(x.x, base, step, e);
        x.y = biased(x.y, base, step, e + 1);
      }
      s[e] = x.x;
      s[e + 1] = x.y;
    }
  });
}

// Rows [r0, 128) of a 128-row operand tile in shared memory (d / 64 halves of 128-byte rows; the
// swizzle moves bytes within a row only) set to zero by one warp, before the tensor cores read
// them: what the memory behind a sequence holds may be NaN, and 0 * NaN is not 0.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0) {
  const int lane = threadIdx.x % 32;
#pragma unroll 1
  for (int r = r0 + lane / 8; r < 128; r += 4)
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh)
      *reinterpret_cast<uint4*>(tile + hh * 128 * 128 + r * 128 + (lane % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace fa
