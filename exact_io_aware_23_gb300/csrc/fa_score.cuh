// Scores that are capped by a tanh and lowered by a bias linear in distance (fa_score_mod): the
// arithmetic that the forward, both passes of the backward and the paged kernel share.
//
//     y = cap * tanh(u / cap) - slope |i - j|,  u = scale * (q . k);   dy/du = 1 - tanh^2(u / cap)
//
// All in the log2 domain, as the softmax is.  The tanh is what costs: through the exponential,
// 1 - 2 / (1 + exp 2x), it takes two more special-function operations a score beside the softmax's
// one, and that unit (16 a clock on an SM) then sets the pace.  Scores well below the cap are the
// common case, so where no score of a warp's tile exceeds 0.4 of the cap, tanh(x) = x P(x^2) with P
// of degree 3 (minimax for the relative error on |x| <= 0.4, found by exchange: 9.9e-8, less than
// two roundings of fp32), five multiply-adds a score; else the exponential form, for the whole tile.
// (B1 H16 Hkv4 N8192 d128 causal, softcap 50: forward 296 us and backward 939 with scores of
// deviation 2, all below 0.4 of the cap; 472 and 1281 with deviation 12, where nearly every tile has
// one beyond it.  Each multiply-add costs 16 us of the forward: degree 4 would reach to 0.6 of the
// cap, degree 6 to the cap itself.)
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "fa_internal.cuh"
#include "ptx_sm103.cuh"

namespace fa {

// P's coefficients, ascending, and its range
constexpr double kTanhPoly[4] = {0.999999901900935, -0.3333136245895285, 0.13270976759047418,
                                 -0.04755360362774448};
constexpr double kTanhRange = 0.4;
// The bf16 backward rebuilds P to round it, and dS, to 8 bits (2^-9 on average 1.7e-3): there degree 2
// does, off by 6.3e-6 of a score, for scores up to 40, 2.5e-4 of P.  (fp16 keeps degree 3.)
constexpr double kTanhLow[3] = {0.999993753137338, -0.33262579481744287, 0.12127786695232969};
constexpr double kLowMost = 40.0;

// Fills the kernels' form of the score arguments for raw products q . k; false when the cap is out
// of the range fp32 can hold them in.
inline bool make_score(const fa_score_mod* m, float scale, ScoreArgs* out) {
  *out = ScoreArgs{};
  if (m == nullptr) return true;
  out->slopes = m->alibi_slopes;
  out->prefix = m->prefix_lens;
  if (m->softcap > 0.f) {
    const double r = (double)scale / (double)m->softcap, cap = (double)m->softcap * 1.4426950408889634;
    out->cap_log2 = (float)cap;
    out->c_exp = (float)(2.0 * r * 1.4426950408889634);
    if (!isfinite(out->cap_log2) || !isfinite(out->c_exp) || !(out->cap_log2 > 0.f)) return false;
    out->poly_limit = (float)(kTanhRange / r);
    if (!isfinite(out->poly_limit)) out->poly_limit = 3.4e38f;
    out->low_limit = (float)fmin((double)out->poly_limit, kLowMost / (double)scale);
    auto twice = [&](double v) {
      const float f = (float)v;
      if (!isfinite(f)) out->poly_limit = out->low_limit = -1.f;    // a tiny cap: always the exponential
      uint32_t bits;
      memcpy(&bits, &f, 4);
      return (uint64_t)bits << 32 | bits;
    };
    double p = r;
    for (int i = 0; i < 4; ++i, p *= r * r) {
      out->poly[i] = twice(kTanhPoly[i] * p);
      out->capped[i] = twice(kTanhPoly[i] * p * cap);
      if (i < 3) out->poly_low[i] = twice(kTanhLow[i] * p);
    }
  }
  return true;
}

// P(z) for two values
template <int N>
__device__ __forceinline__ float2 poly2(float2 z, const uint64_t (&c)[N]) {
  uint64_t zz, p = c[N - 1];
  asm("mov.b64 %0, {%1, %2};" : "=l"(zz) : "f"(z.x), "f"(z.y));
#pragma unroll
  for (int i = N - 2; i >= 0; --i) asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(p), "l"(zz), "l"(c[i]));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
// tanh(scale s / cap) of two raw products within the polynomial's range
__device__ __forceinline__ float2 tanh_poly(float2 s, const ScoreArgs& k) {
  return ptx::mul2(poly2(ptx::mul2(s, s), k.poly), s);
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + exp 2x) for any s; the exponential may overflow to infinity.  tanh = 1 - 2 times this.
__device__ __forceinline__ float2 logistic(float2 s, const ScoreArgs& k) {
  return make_float2(rcp(1.f + ptx::ex2(s.x * k.c_exp)), rcp(1.f + ptx::ex2(s.y * k.c_exp)));
}
__device__ __forceinline__ float2 tanh_exp(float2 s, const ScoreArgs& k) {
  return ptx::fma2(logistic(s, k), make_float2(-2.f, -2.f), make_float2(1.f, 1.f));
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

// The forms of one tile's scores: which tanh, and which bias.
enum : int { kCapNone = 0, kCapPoly = 1, kCapExp = 2 };
enum : int { kBiasNone = 0, kBiasLinear = 1, kBiasAbs = 2 };
// ... as the backward takes it, by the degree that its operands' type F16 asks for
template <int kCap, bool F16>
__device__ __forceinline__ float2 tanh_of(float2 s, const ScoreArgs& k) {
  if constexpr (kCap == kCapExp) return tanh_exp(s, k);
  else if constexpr (F16) return tanh_poly(s, k);
  else return ptx::mul2(poly2(ptx::mul2(s, s), k.poly_low), s);
}
// The bias -slope |i - j| over one thread's row (or column) of a tile, whose distances run on by one:
// at score e it is step * (first + e) where the tile lies on one side of the diagonal (or the other
// side is masked), and step * |first + e| where it crosses it.  `first` is j - i, or i - j, at the
// first score; lo and hi bound it over the unmasked part of the whole tile.  The distance is exact
// before it meets the slope: step * first taken out of the row would round at up to 127 steps, and a
// slope of 1000 move the scores next to the diagonal by 0.01.
struct Bias {
  float first, step;
  bool crosses;
};
__device__ __forceinline__ Bias make_bias(float slope, int first, int lo, int hi) {
  return Bias{(float)first, lo < 0 && hi <= 0 ? slope : -slope, lo < 0 && hi > 0};
}
// Scores e and e + 1 (e even and a constant) with their bias.  The first 16 scores' distances are
// single additions, the others' run on from them in pairs: one packed addition for two scores.
// (Single additions throughout: forward of B1 H16 Hkv4 N8192 d128 causal with cap and bias 382 us
// against 364, backward 1045 against 1030.)
template <int kBias>
__device__ __forceinline__ float2 biased(float2 x, const Bias& b, int e) {
  float2 d = make_float2(b.first + (float)(e & 14), b.first + (float)((e & 14) + 1));
#pragma unroll
  for (int i = 16; i <= e; i += 16) d = ptx::add2(d, make_float2(16.f, 16.f));
  if constexpr (kBias == kBiasAbs) d = make_float2(fabsf(d.x), fabsf(d.y));
  return ptx::fma2(d, make_float2(b.step, b.step), x);
}

// What a call modifies, as the backward's kernels are compiled for it: one kernel for all kinds keeps
// every kind's registers live and spills (B1 H16 Hkv4 N8192 d128 causal with a prefix alone, dK, dV
// and dQ: 799 us by the kernel of all kinds, 748 by its own; with softcap 50, 949 and 930).
enum : int { kModNone = 0, kModCap = 1, kModBias = 2, kModBoth = 3, kModPrefix = 4 };
__host__ inline int mod_of(const ScoreArgs& k) {
  const int m = (k.cap_log2 != 0.f ? kModCap : 0) | (k.slopes != nullptr ? kModBias : 0);
  return m != 0 ? m : kModPrefix;
}

// Calls body(cap form, bias form) as compile-time constants, the same ones in the warp.
template <int V> struct Const { static constexpr int value = V; };
template <int kMod, int N, typename Body>
__device__ __forceinline__ void with_score(const float (&s)[N], const ScoreArgs& k, float limit, const Bias& b,
                                           Body&& body) {
  auto with_cap = [&](auto cap) {
    if constexpr ((kMod & kModBias) == 0) {
      body(cap, Const<kBiasNone>());
    } else {
      if (!b.crosses) body(cap, Const<kBiasLinear>());
      else body(cap, Const<kBiasAbs>());
    }
  };
  if constexpr ((kMod & kModCap) == 0) {
    with_cap(Const<kCapNone>());
  } else {
    if (poly_fits(s, limit)) with_cap(Const<kCapPoly>());
    else with_cap(Const<kCapExp>());
  }
}

// Scores s[0..N) of one row turned into the log2 domain in place.
template <int N>
__device__ __forceinline__ void score_row(float (&s)[N], const ScoreArgs& k, float c, const Bias& b) {
  auto body = [&](auto cap, auto bias) {
    constexpr int kCap = decltype(cap)::value, kBias = decltype(bias)::value;
    const float m = kCap == kCapNone ? c : kCap == kCapPoly ? 1.f : -2.f * k.cap_log2;
    const float a = kCap == kCapExp ? k.cap_log2 : 0.f;
    const float2 m2 = make_float2(m, m), a2 = make_float2(a, a);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      float2 x = make_float2(s[e], s[e + 1]);
      if constexpr (kCap == kCapPoly) x = ptx::mul2(poly2(ptx::mul2(x, x), k.capped), x);
      else if constexpr (kCap == kCapExp) x = ptx::fma2(logistic(x, k), m2, a2);
      else x = ptx::mul2(x, m2);
      if constexpr (kBias != kBiasNone) x = biased<kBias>(x, b, e);
      s[e] = x.x;
      s[e + 1] = x.y;
    }
  };
  if (k.slopes == nullptr) with_score<kModCap>(s, k, k.poly_limit, b, body);
  else if (k.cap_log2 == 0.f) with_score<kModBias>(s, k, k.poly_limit, b, body);
  else with_score<kModBoth>(s, k, k.poly_limit, b, body);
}

// Rows [r0, kRows) of an operand tile in shared memory (d / 64 halves of 128-byte rows; the swizzle
// moves bytes within a row only) set to zero by one warp, before the tensor cores read them: what
// the memory behind a sequence holds may be NaN, and 0 * NaN is not 0.
template <int D, int kRows = 128>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0) {
  const int lane = threadIdx.x % 32;
#pragma unroll 1
  for (int r = r0 + lane / 8; r < kRows; r += 4)
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh)
      *reinterpret_cast<uint4*>(tile + hh * kRows * 128 + r * 128 + (lane % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace fa
