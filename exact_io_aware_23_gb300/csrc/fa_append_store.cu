// The write of new tokens into 8-bit pages, and into pages whose key bounds are kept.
//
// All new tokens of a page and head share what is computed for it, so the work goes by pages: a team (a
// warp for a few new tokens, a block for many) takes one page of one sequence and walks over heads.
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

#include "fa_paged.cuh"
#include "fa_rotate.cuh"
#include "fa_sm103.cuh"
#include "fa_store.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kHold = 2;                   // rows of 16 values that a thread keeps between the two passes

template <typename T>
__device__ __forceinline__ void round_values(float (&x)[8]) {
  Raw8<T> r;
  pack(x, r);
  unpack(r, x);
}

// 16 codes of a row, as they lie in memory
template <int kStore>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  if constexpr (kStore == FA_PAGES_INT8) {
    int i[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) i[e] = __float2int_rn(x[e] * inv);
    return make_uint2(pack_s8(i[0], i[1], i[2], i[3]), pack_s8(i[4], i[5], i[6], i[7]));
  } else {
    return make_uint2(pack_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      pack_e4m3(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
  }
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

// x times a power of two, rounded down, also where the product is below fp32's range
__device__ __forceinline__ int down(float x, float by) {
  const int i = __float2int_rd(x * by);
  return x < 0.f ? min(i, -1) : i;
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
  const int size = a.cache.page_size, lead = max(w->begin, 0) / size + p;
  const int64_t start = (int64_t)lead * size;
  if (count == 0 || start >= len) return false;
  w->first = max(max(w->begin, 0), (int)start);
  w->n = (int)min((int64_t)len, start + size) - w->first;
  w->kept = w->first - (int)start;
  w->page = a.cache.table[b * a.cache.table_stride + lead];
  if ((uint64_t)w->page >= (uint64_t)a.cache.n_pages) {        // reported, not followed
    atomicExch(a.err, kDevBadOffsets);
    return false;
  }
  return true;
}

template <typename T, int kStore, int kTeam>
__device__ __forceinline__ void write_page(const AppendArgs& a, const StoreArgs& st, const PageWork& w, int b, int h0,
                                           int h1, uint32_t* amax_smem, float (*bound_smem)[2][128]) {
  constexpr bool k8 = kStore != FA_PAGES_16BIT;
  const int lt = threadIdx.x % kTeam;
  const int units = a.d / kUnit, rows = kTeam / units;
  const int u = lt % units, r = lt / units;
  const Unit t = unit_of(u, a.rot);
  const bool turns = t.turns && h0 < a.Hkv;
  const int iters = (w.n + rows - 1) / rows;
  uint64_t frac[8];
  float c[kHold][8], s[kHold][8];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) frac[i] = turn_fraction(a.rot.inv_freq[8 * u + i]);
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (i < iters) angles(frac, w.first + i * rows + r, a.rot, c[i], s[i]);
  }
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const bool is_k = h < a.Hkv;
    const int g = is_k ? h : h - a.Hkv;
    const Strides sd = is_k ? a.ks : a.vs;
    const T* const src = static_cast<const T*>(is_k ? a.k : a.v) + b * sd.b + g * sd.h + (int64_t)(w.first - w.begin) * sd.n;
    float* const scales = is_k ? st.k_scales : st.v_scales;
    const int64_t place = w.page * a.Hkv + g;
    float old = 0.f, old_unit = 0.f;
    if (k8 && w.kept > 0) old = scales[place];
    const bool bounds = is_k && st.bounds != nullptr;
    if (bounds && w.kept > 0) old_unit = st.bound_scales[place];

    // a row's 16 values: read, turned
    auto row = [&](int i, float (&x)[8], float (&y)[8], bool held) {
      const T* p = src + (int64_t)(i * rows + r) * sd.n;
      const Raw8<T> lo = load8(p + t.lo), hi = load8(p + t.hi);
      unpack(lo, x);
      unpack(hi, y);
      if (turns && is_k) {
        if (held) {
          turn8(x, y, a.rot.interleaved, c[i < kHold ? i : 0], s[i < kHold ? i : 0]);
        } else {
          float cc[8], ss[8];
          angles(frac, w.first + i * rows + r, a.rot, cc, ss);
          turn8(x, y, a.rot.interleaved, cc, ss);
        }
        if (!k8) {                                       // 16-bit pages: bounds of what is stored
          round_values<T>(x);
          round_values<T>(y);
        }
      }
    };
    float x[kHold][8], y[kHold][8];
    uint32_t amax = 0;
    float mn[2][8], mx[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mn[0][e] = mn[1][e] = INFINITY;
      mx[0][e] = mx[1][e] = -INFINITY;
    }
    auto look = [&](const float (&x)[8], const float (&y)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = max(amax, max(abs_bits(x[e]), abs_bits(y[e])));
      if (bounds) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          mn[0][e] = fminf(mn[0][e], x[e]);
          mx[0][e] = fmaxf(mx[0][e], x[e]);
          mn[1][e] = fminf(mn[1][e], y[e]);
          mx[1][e] = fmaxf(mx[1][e], y[e]);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (i * rows + r < w.n) {
        row(i, x[i], y[i], true);
        look(x[i], y[i]);
      }
    for (int i = kHold; i < iters; ++i)
      if (i * rows + r < w.n) {
        float xx[8], yy[8];
        row(i, xx, yy, false);
        look(xx, yy);
      }

    // the team's largest value and bounds
    if (k8 || bounds) {
      amax = __reduce_max_sync(0xffffffffu, amax);
      if (bounds) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float& lo = mn[e / 8][e % 8];
          float& hi = mx[e / 8][e % 8];
          for (int o = 16; o >= units; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
          }
        }
      }
      if constexpr (kTeam > 32) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        if (lane == 0) amax_smem[warp] = amax;
        if (bounds && lane < units) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            bound_smem[warp][0][t.lo + e] = mn[0][e];
            bound_smem[warp][0][t.hi + e] = mn[1][e];
            bound_smem[warp][1][t.lo + e] = mx[0][e];
            bound_smem[warp][1][t.hi + e] = mx[1][e];
          }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTeam / 32; ++i) amax = max(amax, amax_smem[i]);
        if (bounds && lt < units) {
#pragma unroll 1
          for (int i = 1; i < kTeam / 32; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              mn[0][e] = fminf(mn[0][e], bound_smem[i][0][t.lo + e]);
              mn[1][e] = fminf(mn[1][e], bound_smem[i][0][t.hi + e]);
              mx[0][e] = fmaxf(mx[0][e], bound_smem[i][1][t.lo + e]);
              mx[1][e] = fmaxf(mx[1][e], bound_smem[i][1][t.hi + e]);
            }
        }
      }
      __syncwarp();
    }
    const bool finite = amax < 0x7f800000u;

    // codes
    typename StoredAs<T, kStore>::type* const dst =
        static_cast<typename StoredAs<T, kStore>::type*>(is_k ? a.cache.k : a.cache.v) + w.page * a.cache.page_stride +
        g * a.cache.head_stride;
    float inv = 0.f, scale = 0.f;
    if constexpr (k8) {
      const float need = finite ? power_scale<kStore == FA_PAGES_INT8>(amax) : __uint_as_float(0x7fc00000u);
      scale = old != old || need != need ? __uint_as_float(0x7fc00000u) : fmaxf(old, need);
      inv = scale == scale ? 1.f / scale : 0.f;
    }
    auto store = [&](int i, float (&x)[8], float (&y)[8]) {
      auto* p = dst + (int64_t)(w.kept + i * rows + r) * a.cache.token_stride;
      if constexpr (k8) {
        if (scale != scale) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
        }
        *reinterpret_cast<uint2*>(p + t.lo) = encode8<kStore>(x, inv);
        *reinterpret_cast<uint2*>(p + t.hi) = encode8<kStore>(y, inv);
      } else {
        Raw8<T> lo, hi;
        pack(x, lo);
        pack(y, hi);
        store8(p + t.lo, lo);
        store8(p + t.hi, hi);
      }
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (i * rows + r < w.n) store(i, x[i], y[i]);
    for (int i = kHold; i < iters; ++i)
      if (i * rows + r < w.n) {
        float xx[8], yy[8];
        row(i, xx, yy, false);
        store(i, xx, yy);
      }
    if constexpr (k8) {
      if (w.kept > 0 && scale > old) {                  // (not where either is NaN)
        const float ratio = old / scale;
        for (int i = r; i < w.kept; i += rows) {
          uint4* p = reinterpret_cast<uint4*>(dst + (int64_t)i * a.cache.token_stride + kUnit * u);
          uint4 v = *p;
          v.x = recode<kStore>(v.x, ratio);
          v.y = recode<kStore>(v.y, ratio);
          v.z = recode<kStore>(v.z, ratio);
          v.w = recode<kStore>(v.w, ratio);
          *p = v;
        }
      }
      if (lt == 0) scales[place] = scale;
    }
    if (bounds && lt < units) {
      const float need = finite ? power_scale<true>(amax) : __uint_as_float(0x7fc00000u);
      const float unit = old_unit != old_unit || need != need ? __uint_as_float(0x7fc00000u) : fmaxf(old_unit, need);
      const float by = unit == unit ? 1.f / unit : 0.f, ratio = w.kept > 0 && unit == unit ? old_unit / unit : 0.f;
      int8_t* const q = st.bounds + place * 2 * a.d;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int at = half == 0 ? t.lo : t.hi;
        int lo[8], hi[8];
        uint2* const plo = reinterpret_cast<uint2*>(q + at);
        uint2* const phi = reinterpret_cast<uint2*>(q + a.d + at);
        const uint2 was_lo = w.kept > 0 ? *plo : make_uint2(0u, 0u), was_hi = w.kept > 0 ? *phi : make_uint2(0u, 0u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo[e] = down(mn[half][e], by);
          hi[e] = -down(-mx[half][e], by);
          if (w.kept > 0) {
            lo[e] = min(lo[e], down((float)(int8_t)((e < 4 ? was_lo.x : was_lo.y) >> (8 * (e & 3))), ratio));
            hi[e] = max(hi[e], -down(-(float)(int8_t)((e < 4 ? was_hi.x : was_hi.y) >> (8 * (e & 3))), ratio));
          }
        }
        *plo = make_uint2(pack_s8(lo[0], lo[1], lo[2], lo[3]), pack_s8(lo[4], lo[5], lo[6], lo[7]));
        *phi = make_uint2(pack_s8(hi[0], hi[1], hi[2], hi[3]), pack_s8(hi[4], hi[5], hi[6], hi[7]));
      }
      if (lt == 0) st.bound_scales[place] = unit;
    }
    if constexpr (kTeam > 32) __syncthreads();           // the shared words are written again
  }
}

// Queries: turned and copied, as in the write into 16-bit pages.
template <typename T>
__device__ __forceinline__ void turn_queries(const AppendArgs& a, const StoreArgs& st, int64_t block) {
  constexpr int kBatch = 4;
  const int units = a.d / kUnit, per_block = kThreads / units;
  const int u = threadIdx.x % units;
  const Unit t = unit_of(u, a.rot);
  const int h0 = (int)(block % st.q_head_blocks) * st.q_heads, h1 = min(a.H, h0 + st.q_heads);
  const int64_t m = block / st.q_head_blocks * per_block + threadIdx.x / units;
  if (m >= (int64_t)a.B * a.T) return;
  const int b = (int)(m / a.T), n = (int)(m % a.T);
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

template <typename T, int kStore, int kTeam>
__global__ void __launch_bounds__(kThreads) append_store_kernel(const AppendArgs a, const StoreArgs st) {
  __shared__ uint32_t amax_smem[kThreads / 32];
  __shared__ float bound_smem[kTeam > 32 ? kThreads / 32 : 1][2][128];
  if ((int64_t)blockIdx.x >= st.page_blocks) {
    turn_queries<T>(a, st, (int64_t)blockIdx.x - st.page_blocks);
    return;
  }
  const int64_t team = (int64_t)blockIdx.x * (kThreads / kTeam) + threadIdx.x / kTeam;
  const int64_t bp = team / st.head_blocks;
  const int h0 = (int)(team % st.head_blocks) * st.heads, h1 = min(2 * a.Hkv, h0 + st.heads);
  const int b = (int)(bp / st.span), p = (int)(bp % st.span);
  PageWork w;
  if (b >= a.B || !page_work(a, b, p, &w)) return;
  write_page<T, kStore, kTeam>(a, st, w, b, h0, h1, amax_smem, bound_smem);
}

template <typename T, int kStore>
cudaError_t append_store(const AppendArgs& a, StoreArgs st, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int units = a.d / kUnit;
  st.span = (a.T + a.cache.page_size - 2) / a.cache.page_size + 1;
  // a warp holds kHold * 32 / units tokens' rows
  const bool warps = a.T <= kHold * 32 / units;
  const int64_t pages = (int64_t)a.B * st.span;
  st.heads = 2 * a.Hkv;
  if (warps) st.heads = 1;
  else
    while (st.heads > 1 && pages * ((2 * a.Hkv + st.heads - 1) / st.heads) < 4 * sms) st.heads = (st.heads + 1) / 2;
  st.head_blocks = (2 * a.Hkv + st.heads - 1) / st.heads;
  const int per = warps ? kThreads / 32 : 1;
  st.page_blocks = (pages * st.head_blocks + per - 1) / per;
  int64_t q_blocks = 0;
  if (a.q != nullptr) {
    const int64_t tokens = ((int64_t)a.B * a.T + kThreads / units - 1) / (kThreads / units);
    st.q_heads = a.H;
    while (st.q_heads > 4 && tokens * ((a.H + st.q_heads - 1) / st.q_heads) < 4 * sms) st.q_heads = (st.q_heads + 1) / 2;
    st.q_head_blocks = (a.H + st.q_heads - 1) / st.q_heads;
    q_blocks = tokens * st.q_head_blocks;
  }
  const int64_t grid = st.page_blocks + q_blocks;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (warps) append_store_kernel<T, kStore, 32><<<(unsigned)grid, kThreads, 0, s>>>(a, st);
  else append_store_kernel<T, kStore, kThreads><<<(unsigned)grid, kThreads, 0, s>>>(a, st);
  return cudaGetLastError();
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
