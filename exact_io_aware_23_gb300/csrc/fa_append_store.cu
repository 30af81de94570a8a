// The write of new tokens into 8-bit pages, and into pages whose key bounds are kept.
//
// All new tokens of a page and head share what is computed for it, so the work goes by pages: a team (a
// warp for a few new tokens, a block for many) takes one page of one sequence and one head, of its keys or values.
//
//     amax = max |x| over the page's new tokens,  need = the smallest 2^e, e >= -100, with amax <= largest 2^e
//     scale' = max(scale, need) (need alone where the page held no token before)
//     code = x / scale' rounded to nearest even; codes of earlier tokens times scale / scale' where it grew
//
// Powers of two make every quotient exact, so a code is one rounding of its value whatever the order of
// the writes; and as a growth at least doubles the scale, all later roundings of a code together
// come to less than one step.  (A scale of amax / 127 itself would be up to 2 times finer for int8, and
// no better for e4m3, whose precision goes with the value; but a page of 64 tokens written one by one
// would round its first one again each time that a larger value comes.)  What is not finite makes the
// scale NaN, for as long as the page lives, and so shows in every result that reads it.
//
// Bounds.  The smallest and largest of each of the d values over the page's keys, downwards and upwards to
// whole numbers of their own scale (need with 127): they grow with the page in the same way.
//
// What bounds it: bytes, two read and one written a value, and for one token a sequence the chain of
// reads: lengths, table entry, scale.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fa_paged.cuh"
#include "fa_rotate.cuh"
#include "fa_sm103.cuh"
#include "fa_store.cuh"

namespace fa {
namespace {

constexpr int kPageRows = 4;               // rows of 16 values that a thread holds

template <typename T>
__device__ __forceinline__ void round_values(float (&x)[8]) {
  Raw8<T> r;
  pack(x, r);
  unpack(r, x);
}

// four codes times a power of two, rounded again
template <int kStore>
__device__ __forceinline__ uint32_t recode(uint32_t c, float ratio) {
  if constexpr (kStore == FA_PAGES_INT8) {
    int i[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) i[e] = __float2int_rn((float)(int8_t)(c >> (8 * e)) * ratio);
    return pack_s8(i[0], i[1], i[2], i[3]);
  } else {
    float f[4];
    unpack_e4m3(c, f);
    return pack_e4m3(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
  }
}

// x / unit rounded down, exactly, for |x| up to 128 of any positive unit; by: 1 / unit, rounded.  What the
// rounded product says is one too much or too little at most, and the signs of remainders, which their one rounding keeps, tell.
__device__ __forceinline__ int down(float x, float unit, float by) {
  const int i = __float2int_rd(x * by);
  return i + (fmaf(-(float)i, unit, x) < 0.f ? -1 : fmaf(-(float)(i + 1), unit, x) >= 0.f ? 1 : 0);
}
// A bound c, in whole numbers of `old`, in those of `unit`, rounded down in the same way.  unit is old or, where it grew, a
// power of two, so that i * unit is exact.
__device__ __forceinline__ int down_again(int c, float old, float unit, float ratio) {
  if (old == unit) return c;
  const int i = __float2int_rd((float)c * ratio);
  return i + (fmaf((float)c, old, -((float)i * unit)) < 0.f ? -1 : fmaf((float)c, old, -((float)(i + 1) * unit)) >= 0.f ? 1 : 0);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A page of one sequence that gets tokens.
struct PageWork {
  int64_t page;               // its place in the cache
  int begin;                  // place of the sequence's first new token
  int first, n;               // the page's first new token's place, and their number
  int kept;                   // tokens that were there before
};
__device__ __forceinline__ bool page_work(const AppendArgs& a, int b, int p, PageWork* w) {
  const int count = new_tokens(a.q_lens, b, a.T);
  const int len = paged_len(a.cache, b, a.err);
  w->begin = len - count;
  const int size = a.cache.page_size, lead = (int)((uint32_t)max(w->begin, 0) / (uint32_t)size) + p;
  const int64_t start = (int64_t)lead * size;
  if (count == 0 || start >= len) return false;
  w->first = max(max(w->begin, 0), (int)start);
  w->n = (int)min((int64_t)len, start + size) - w->first;
  w->kept = w->first - (int)start;
  w->page = a.cache.table[b * a.cache.table_stride + lead];
  return true;
}
// Whether the page exists (asked once the tokens' reads are on their way).
__device__ __forceinline__ bool page_exists(const AppendArgs& a, const PageWork& w) {
  if ((uint64_t)w.page < (uint64_t)a.cache.n_pages) return true;
  atomicExch(a.err, kDevBadOffsets);                           // reported, not followed
  return false;
}

// 16 values of a row as they lie in memory: pairs of 16-bit values, or fp32 where they are turned.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ float2 values(uint32_t x) { return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)); }
};
template <> struct Pair<__half> {
  using type = __half2;
  static __device__ __forceinline__ float2 values(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }
};
template <typename T>
__device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
  using P = typename Pair<T>::type;
  const P r = __hmin2(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
  using P = typename Pair<T>::type;
  const P r = __hmax2(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// the fp32 bits of the larger of two 16-bit values without signs
template <typename T>
__device__ __forceinline__ uint32_t larger_bits(uint32_t x) {
  const uint32_t m = max(x & 0xffffu, x >> 16);
  return __float_as_uint(Pair<T>::values(m).x);
}

// Four values times inv (a power of two's inverse, products within +-127.5) to int8: adding 1.5 * 2^23 rounds
// to a whole number, ties to even, whose low byte is the code.
__device__ __forceinline__ uint32_t quick_s8(float a, float b, float c, float d, float inv) {
  constexpr float kMagic = 12582912.f;
  const uint32_t x = __float_as_uint(fmaf(a, inv, kMagic)), y = __float_as_uint(fmaf(b, inv, kMagic));
  const uint32_t z = __float_as_uint(fmaf(c, inv, kMagic)), w = __float_as_uint(fmaf(d, inv, kMagic));
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}
template <int kStore>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  if constexpr (kStore == FA_PAGES_INT8) return quick_s8(a, b, c, d, inv);
  else return pack_e4m3(a * inv, b * inv, c * inv, d * inv);
}

// A page and head, by a team of kTeam threads (a warp, or the block), each of which holds kPageRows rows of 16 values:
// a warp 16 tokens of d = 128, or 32 of d = 64, 128 threads four times as many.  Several blocks share an SM, so
// one's barrier and writes hide behind the others' reads.  Pages of more tokens than the team holds are read
// twice.  kTurn: key heads are turned (value heads take the path of 16-bit values).
template <typename T, int kStore, bool kTurn, bool kBounds, int kTeam>
__device__ __forceinline__ void write_page(const AppendArgs& a, const StoreArgs& st, int b, int p, int h, uint32_t* smem) {
  constexpr bool k8 = kStore != FA_PAGES_16BIT;
  constexpr int kWarps = kTeam / 32, kRows = kPageRows;
  uint32_t* const bound_smem = smem;                       // [2][kWarps][d], or of pairs
  uint32_t* const amax_smem = smem + (kBounds ? 2 * kWarps * (kTurn ? 128 : 64) : 0);   // [kWarps]
  const int mine = threadIdx.x % kTeam, warp = mine / 32, lane = mine % 32;
  const int units = a.d / kUnit, rows = kTeam / units;
  const int u = mine % units, r = mine / units;
  const Unit t = kTurn ? unit_of(u, a.rot) : Unit{kUnit * u, kUnit * u + 8, false};
  const bool is_k = h < a.Hkv;
  const int g = is_k ? h : h - a.Hkv;
  PageWork w;
  if (!page_work(a, b, p, &w)) return;
  const Strides sd = is_k ? a.ks : a.vs;
  const T* const src = static_cast<const T*>(is_k ? a.k : a.v) + b * sd.b + g * sd.h + (int64_t)(w.first - w.begin) * sd.n;
  const int64_t place = w.page * a.Hkv + g;
  float* const scales = is_k ? st.k_scales : st.v_scales;
  const bool bounds = kBounds && is_k;

  // a row: eight pairs of 16-bit values, or 16 values in fp32
  using Word = std::conditional_t<kTurn, float, uint32_t>;
  constexpr int kWords = kTurn ? 16 : 8;
  uint64_t frac[kTurn ? 8 : 1];
  if constexpr (kTurn) {
    if (t.turns) {
#pragma unroll
      for (int i = 0; i < 8; ++i) frac[i] = turn_fraction(a.rot.inv_freq[8 * u + i]);
    }
  }
  auto read = [&](int i, Raw8<T>& lo, Raw8<T>& hi) {
    const T* q = src + (int64_t)(i * rows + r) * sd.n;
    lo = load8(q + t.lo);
    hi = load8(q + t.hi);
  };
  auto take = [&](int i, const Raw8<T>& lo, const Raw8<T>& hi, Word (&x)[kWords]) {
    if constexpr (kTurn) {
      float p0[8], p1[8];
      unpack(lo, p0);
      unpack(hi, p1);
      if (t.turns) {
        float c[8], s[8];
        angles(frac, w.first + i * rows + r, a.rot, c, s);
        turn8(p0, p1, a.rot.interleaved, c, s);
        if (!k8) {                                         // 16-bit pages: bounds of what is stored
          round_values<T>(p0);
          round_values<T>(p1);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = p0[e];
        x[8 + e] = p1[e];
      }
    } else {
      const uint32_t v[8] = {lo.w[0].x, lo.w[0].y, lo.w[0].z, lo.w[0].w, hi.w[0].x, hi.w[0].y, hi.w[0].z, hi.w[0].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v[e];
    }
  };
  uint32_t amax = 0;
  Word mn[kBounds ? kWords : 1], mx[kBounds ? kWords : 1];
  bool any = false;
  auto look = [&](const Word (&x)[kWords]) {
#pragma unroll
    for (int e = 0; e < kWords; ++e) {
      if constexpr (kTurn) amax = max(amax, abs_bits(x[e]));
      else amax = max_u16x2(amax, x[e] & 0x7fff7fffu);
    }
    if constexpr (kBounds) {
      if (bounds) {
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
          if constexpr (kTurn) {
            mn[e] = any ? fminf(mn[e], x[e]) : x[e];
            mx[e] = any ? fmaxf(mx[e], x[e]) : x[e];
          } else {
            mn[e] = any ? least<T>(mn[e], x[e]) : x[e];
            mx[e] = any ? most<T>(mx[e], x[e]) : x[e];
          }
        }
        any = true;
      }
    }
  };
  Word x[kRows][kWords];
  {
    Raw8<T> lo[kRows], hi[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i * rows + r < w.n) read(i, lo[i], hi[i]);
    if (!page_exists(a, w)) return;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i * rows + r < w.n) {
        take(i, lo[i], hi[i], x[i]);
        look(x[i]);
      }
  }
  for (int i = kRows; i * rows + r < w.n; ++i) {
    Raw8<T> lo, hi;
    Word y[kWords];
    read(i, lo, hi);
    take(i, lo, hi, y);
    look(y);
  }
  float old = 0.f, old_unit = 0.f;
  if (k8 && w.kept > 0) old = scales[place];
  if (bounds && w.kept > 0) old_unit = st.bound_scales[place];

  // the page's largest value, and its bounds
  if constexpr (!kTurn) amax = larger_bits<T>(amax);
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (lane == 0) amax_smem[warp] = amax;
  if constexpr (kBounds) {
    if (bounds) {
      // threads without a row: +inf, -inf
      const uint32_t inf = kTurn ? 0x7f800000u : std::is_same_v<T, __half> ? 0x7c007c00u : 0x7f807f80u;
      const uint32_t sign = kTurn ? 0x80000000u : 0x80008000u;
#pragma unroll
      for (int e = 0; e < kWords; ++e) {
        if constexpr (kTurn) {
          mn[e] = any ? mn[e] : __uint_as_float(inf);
          mx[e] = any ? mx[e] : __uint_as_float(inf | sign);
        } else {
          mn[e] = any ? mn[e] : inf;
          mx[e] = any ? mx[e] : inf | sign;
        }
        for (int o = 16; o >= units; o >>= 1) {
          if constexpr (kTurn) {
            mn[e] = fminf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], o));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
          } else {
            mn[e] = least<T>(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], o));
            mx[e] = most<T>(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
          }
        }
      }
      if (lane < units) {
        const int words = kTurn ? a.d : a.d / 2;
        uint32_t* const lo = bound_smem + warp * words;
        uint32_t* const hi = lo + kWarps * words;
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
          const int at = kTurn ? (e < 8 ? t.lo + e : t.hi + e - 8) : 8 * u + e;
          lo[at] = reinterpret_cast<const uint32_t&>(mn[e]);
          hi[at] = reinterpret_cast<const uint32_t&>(mx[e]);
        }
      }
    }
  }
  if constexpr (kTeam > 32) __syncthreads();
  else __syncwarp();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) amax = max(amax, amax_smem[i]);
  const bool finite = amax < 0x7f800000u;

  // codes
  using Elem = typename StoredAs<T, kStore>::type;
  Elem* const dst = static_cast<Elem*>(is_k ? a.cache.k : a.cache.v) + w.page * a.cache.page_stride + g * a.cache.head_stride;
  float inv = 0.f, scale = 0.f;
  if constexpr (k8) {
    const float need = finite ? power_scale<kStore == FA_PAGES_INT8>(amax) : __uint_as_float(0x7fc00000u);
    scale = old != old || need != need ? __uint_as_float(0x7fc00000u) : fmaxf(old, need);
    inv = 1.f / scale;
  }
  auto store = [&](int i, const Word (&x)[kWords]) {
    Elem* const q = dst + (int64_t)(w.kept + i * rows + r) * a.cache.token_stride;
    if constexpr (k8) {
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (kTurn) {
          c[e] = encode4<kStore>(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3], inv);
        } else {
          const float2 y = Pair<T>::values(x[2 * e]), z = Pair<T>::values(x[2 * e + 1]);
          c[e] = encode4<kStore>(y.x, y.y, z.x, z.y, inv);
        }
        if (scale != scale) c[e] = 0u;
      }
      if constexpr (kTurn) {
        *reinterpret_cast<uint2*>(q + t.lo) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2*>(q + t.hi) = make_uint2(c[2], c[3]);
      } else {
        *reinterpret_cast<uint4*>(q + t.lo) = make_uint4(c[0], c[1], c[2], c[3]);
      }
    } else if constexpr (kTurn) {
      float p0[8], p1[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p0[e] = x[e];
        p1[e] = x[8 + e];
      }
      Raw8<T> lo, hi;
      pack(p0, lo);
      pack(p1, hi);
      store8(q + t.lo, lo);
      store8(q + t.hi, hi);
    } else {
      *reinterpret_cast<uint4*>(q + t.lo) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(q + t.hi) = make_uint4(x[4], x[5], x[6], x[7]);
    }
  };
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (i * rows + r < w.n) store(i, x[i]);
  for (int i = kRows; i * rows + r < w.n; ++i) {
    Raw8<T> lo, hi;
    Word y[kWords];
    read(i, lo, hi);
    take(i, lo, hi, y);
    store(i, y);
  }
  if constexpr (k8) {
    if (w.kept > 0 && scale > old) {                       // (not where either is NaN)
      const float ratio = old / scale;
      for (int i = r; i < w.kept; i += rows) {
        uint4* q = reinterpret_cast<uint4*>(dst + (int64_t)i * a.cache.token_stride + kUnit * u);
        uint4 v = *q;
        v.x = recode<kStore>(v.x, ratio);
        v.y = recode<kStore>(v.y, ratio);
        v.z = recode<kStore>(v.z, ratio);
        v.w = recode<kStore>(v.w, ratio);
        *q = v;
      }
    }
    if (mine == 0) scales[place] = scale;
  }
  if constexpr (kBounds) {
    if (bounds) {
      const int words = kTurn ? a.d : a.d / 2;
      const float need = finite ? power_scale<true>(amax) : __uint_as_float(0x7fc00000u);
      const float unit = old_unit != old_unit || need != need ? __uint_as_float(0x7fc00000u) : fmaxf(old_unit, need);
      const float by = unit == unit ? 1.f / unit : 0.f, ratio = w.kept > 0 && unit == unit ? old_unit / unit : 0.f;
      for (int x = mine; x < a.d / 2; x += kTeam) {        // two of the d values at a time
        float lo[2], hi[2];
#pragma unroll 1
        for (int i = 0; i < kWarps; ++i) {
          const uint32_t* const q = bound_smem + i * words;
          float2 l, m;
          if constexpr (kTurn) {
            l = reinterpret_cast<const float2*>(q)[x];
            m = reinterpret_cast<const float2*>(q + kWarps * words)[x];
          } else {
            l = Pair<T>::values(q[x]);
            m = Pair<T>::values(q[kWarps * words + x]);
          }
          lo[0] = i == 0 ? l.x : fminf(lo[0], l.x);
          lo[1] = i == 0 ? l.y : fminf(lo[1], l.y);
          hi[0] = i == 0 ? m.x : fmaxf(hi[0], m.x);
          hi[1] = i == 0 ? m.y : fmaxf(hi[1], m.y);
        }
        char2* const q = reinterpret_cast<char2*>(st.bounds + place * 2 * a.d) + x;
        int c[4] = {down(lo[0], unit, by), down(lo[1], unit, by), -down(-hi[0], unit, by), -down(-hi[1], unit, by)};
        if (w.kept > 0) {
          const char2 was_lo = q[0], was_hi = q[a.d / 2];
          c[0] = min(c[0], down_again(was_lo.x, old_unit, unit, ratio));
          c[1] = min(c[1], down_again(was_lo.y, old_unit, unit, ratio));
          c[2] = max(c[2], -down_again(-was_hi.x, old_unit, unit, ratio));
          c[3] = max(c[3], -down_again(-was_hi.y, old_unit, unit, ratio));
        }
        const uint32_t packed = pack_s8(c[0], c[1], c[2], c[3]);
        q[0] = make_char2((signed char)packed, (signed char)(packed >> 8));
        q[a.d / 2] = make_char2((signed char)(packed >> 16), (signed char)(packed >> 24));
      }
      if (mine == 0) st.bound_scales[place] = unit;
    }
  }
}

// Queries: turned and copied, as in the write into 16-bit pages.
template <typename T, int kThr>
__device__ __forceinline__ void turn_queries(const AppendArgs& a, const StoreArgs& st, uint32_t block) {
  constexpr int kBatch = 4;
  const int units = a.d / kUnit, per_block = kThr / units;
  const int u = threadIdx.x % units;
  const Unit t = unit_of(u, a.rot);
  const uint32_t group = block / (uint32_t)st.q_head_blocks;
  const int h0 = (int)(block - group * st.q_head_blocks) * st.q_heads, h1 = min(a.H, h0 + st.q_heads);
  const uint32_t m = group * per_block + threadIdx.x / units;      // (B * T is below 2^31)
  if (m >= (uint32_t)a.B * (uint32_t)a.T) return;
  const int b = (int)(m / (uint32_t)a.T), n = (int)(m - (uint32_t)b * a.T);
  const int count = new_tokens(a.q_lens, b, a.T);
  const int pos = paged_len(a.cache, b, nullptr) - count + n;
  const bool there = n < count && pos >= 0;
  float c[8], s[8];
  if (t.turns && there) {
    uint64_t frac[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) frac[i] = turn_fraction(a.rot.inv_freq[8 * u + i]);
    angles(frac, pos, a.rot, c, s);
  }
  for (int h = h0; h < h1; h += kBatch) {
    Raw8<T> lo[kBatch], hi[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      lo[i] = hi[i] = Raw8<T>{};                         // queries that do not exist: zero
      if (there && h + i < h1) {
        const T* x = static_cast<const T*>(a.q) + b * a.qs.b + (h + i) * a.qs.h + n * a.qs.n;
        lo[i] = load8(x + t.lo);
        hi[i] = load8(x + t.hi);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= h1) break;
      if (t.turns && there) turn_raw(lo[i], hi[i], a.rot.interleaved, c, s);
      T* y = static_cast<T*>(a.q_out) + (((int64_t)b * a.H + h + i) * a.T + n) * a.d;
      store8(y + t.lo, lo[i]);
      store8(y + t.hi, hi[i]);
    }
  }
}

// kThr threads a block, teams of kTeam.  Turned keys take registers: fewer blocks on an SM.  Otherwise as many as there can be,
// though 72 registers spill four words, and six where 8-bit pages have bounds: 4 ragged prompts of up to 4096 tokens at d = 128,
// int8 and bounds, 21.5 us with five blocks, 19.5 with six, 19.1 with seven; without bounds 17.1 with six and 15.6 with seven;
// e4m3 and bounds at d = 64 17.8, 16.3 and 15.6.  Most spilled, 24 words at 128 registers, are those of the warps that turn
// keys for 8-bit pages without bounds (a decoding step): 64 tokens take 5.06 us, and 4.99 with 168 registers and none spilled.
template <typename T, int kStore, bool kTurn, bool kBounds, int kTeam, int kThr>
__global__ void __launch_bounds__(kThr, (kTurn && kBounds ? 384 : kTurn ? 512 : kTeam == 32 && kBounds ? 640 : kTeam == 128 ? 896 : 768) / kThr)
    append_store_kernel(const AppendArgs a, const StoreArgs st) {
  constexpr int kWarps = kTeam / 32, kTeams = kThr / kTeam;
  constexpr int kWords = kWarps + (kBounds ? 2 * kWarps * (kTurn ? 128 : 64) : 0);
  __shared__ __align__(16) uint32_t smem[kTeams][(kWords + 3) / 4 * 4];
  if ((int64_t)blockIdx.x >= st.page_blocks) {
    turn_queries<T, kThr>(a, st, blockIdx.x - (uint32_t)st.page_blocks);
    return;
  }
  // (32 bits: a division in 64 is longer than a row's work)
  const uint32_t team = blockIdx.x * kTeams + threadIdx.x / kTeam, heads = 2u * a.Hkv;
  const uint32_t bp = team / heads, b = bp / (uint32_t)st.span;
  const int h = (int)(team - bp * heads), p = (int)(bp - b * st.span);
  if (b >= (uint32_t)a.B) return;                          // (teams behind the last one: warps)
  uint32_t* const words = smem[threadIdx.x / kTeam];
  if constexpr (kTurn) {
    if (h < a.Hkv) {
      write_page<T, kStore, true, kBounds, kTeam>(a, st, (int)b, p, h, words);
      return;
    }
  }
  write_page<T, kStore, false, kBounds, kTeam>(a, st, (int)b, p, h, words);
}

template <typename T, int kStore, bool kTurn, bool kBounds>
cudaError_t append_store(const AppendArgs& a, StoreArgs st, int sms, cudaStream_t s) {
  constexpr int kLarge = kTurn ? 256 : 512;                // a team of more tokens than 128 threads hold
  const int units = a.d / kUnit;
  st.span = (int)(((int64_t)a.T + a.cache.page_size - 2) / a.cache.page_size) + 1;
  const int64_t heads = (int64_t)a.B * st.span * 2 * a.Hkv;       // of all pages
  // the smallest team that holds the new tokens of any page
  const int most = std::min(a.cache.page_size, a.T);
  const int team = most <= 32 / units * kPageRows ? 32 : most <= 128 / units * kPageRows ? 128 : kLarge;
  const int threads = std::max(team, 128);
  st.page_blocks = (heads + threads / team - 1) / (threads / team);
  int64_t q_blocks = 0;
  if (a.q != nullptr) {
    const int64_t tokens = ((int64_t)a.B * a.T + threads / units - 1) / (threads / units);
    st.q_heads = a.H;
    while (st.q_heads > 4 && tokens * ((a.H + st.q_heads - 1) / st.q_heads) < 1024 * (int64_t)sms / threads)
      st.q_heads = (st.q_heads + 1) / 2;
    st.q_head_blocks = (a.H + st.q_heads - 1) / st.q_heads;
    q_blocks = tokens * st.q_head_blocks;
  }
  if (heads > 0x7fffff00 || st.page_blocks + q_blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)(st.page_blocks + q_blocks);
  if (team == 32) append_store_kernel<T, kStore, kTurn, kBounds, 32, 128><<<grid, 128, 0, s>>>(a, st);
  else if (team == 128) append_store_kernel<T, kStore, kTurn, kBounds, 128, 128><<<grid, 128, 0, s>>>(a, st);
  else append_store_kernel<T, kStore, kTurn, kBounds, kLarge, kLarge><<<grid, kLarge, 0, s>>>(a, st);
  return cudaGetLastError();
}

template <typename T, int kStore>
cudaError_t append_store(const AppendArgs& a, const StoreArgs& st, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (st.bounds != nullptr)
    return a.rot.rot > 0 ? append_store<T, kStore, true, true>(a, st, sms, s) : append_store<T, kStore, false, true>(a, st, sms, s);
  if constexpr (kStore != FA_PAGES_16BIT)
    return a.rot.rot > 0 ? append_store<T, kStore, true, false>(a, st, sms, s) : append_store<T, kStore, false, false>(a, st, sms, s);
  return cudaErrorInvalidValue;                            // 16-bit pages without bounds: launch_append
}

template <typename T>
cudaError_t append_store(const AppendArgs& a, const StoreArgs& st, cudaStream_t s) {
  if (st.store == FA_PAGES_E4M3) return append_store<T, FA_PAGES_E4M3>(a, st, s);
  if (st.store == FA_PAGES_INT8) return append_store<T, FA_PAGES_INT8>(a, st, s);
  return append_store<T, FA_PAGES_16BIT>(a, st, s);
}

}  // namespace

cudaError_t launch_append_store(const AppendArgs& a, const StoreArgs& st, fa_dtype dt, cudaStream_t s) {
  return dt == FA_FP16 ? append_store<__half>(a, st, s) : append_store<__nv_bfloat16>(a, st, s);
}

}  // namespace fa
