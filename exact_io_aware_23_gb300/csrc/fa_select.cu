// The choice of the pages that a sequence's next tokens attend to.
//
// For a query row q and a page whose keys lie between lo and hi in every one of the d values,
//     q . k <= sum_i max(q_i lo_i, q_i hi_i) = 1/2 sum_i (q_i (hi_i + lo_i) + |q_i| (hi_i - lo_i))
// for each of the page's keys.  (Bounds are those of the keys before they go to 8 bits.  Codes of int8 pages keep within
// them, being rounded to the bounds' own whole numbers; one of an e4m3 page can lie outside by its rounding, 2^-4 of a
// value.)  With q in whole numbers of 2^f (8 bits, like lo and hi) all these are whole numbers,
// the operands exact in fp16 and the sum, below 2^23, in fp32, in any order: the choice does not depend on how
// the work is cut up.  A page's score is the largest over the rows of its key head's group of that times 2^f times
// the bounds' scale; the first and the last pages, which are always chosen, and scores that are NaN stand
// above all others, and of equal ones the lower page is chosen.
//
// Scores.  A warp takes 32 pages at a time, their bounds operands of mma.sync as they lie in memory: eight pages the right
// one and 16 rows' q the left one, or with up to 8 rows 16 pages the left one and the rows the right one, half the
// products.  What bounds it: for many pages the warps' own work, 12 instructions a product for sums and differences, and
// DRAM: 64 sequences of 1024 pages, 8 key heads of 4 rows, d = 128, 136 MB, take 36 us with the choice, 3.7 TB/s, and 48
// with products of 16 rows; for few pages the chain of reads: lengths, table entry, bounds.
// Choice.  A block has a (sequence, key head), a slice: it keeps the scores in shared memory and narrows down the range
// of the K-th largest one's bits, 1024 bins at a time.  The bins are laid over the range that the scores
// have: by the bits from the top nearly all would meet in the few bins of their exponents.  What costs there
// is not the bytes but instructions that come from cold caches: loops that are not unrolled, and queries converted once for
// a block, took 64 sequences of up to 128 pages from 10.2 us to 8.6.
// Where there are fewer of them than SMs, and many pages, a kernel of its own scores the pages on all SMs first.
// Few slices: the block that comes last of those that score a slice chooses, in the same launch (two sequences of 8192
// pages and 8 key heads: 23.0 us in two launches, 22.7 in one, one sequence of 1000 pages 10.6 and 9.1; more slices would
// leave some SMs without a block).
// (A cluster of 4 or 8 blocks for each instead, scores in the first one's shared memory: 32 and 36 us for two
// sequences of 8192 pages and 8 key heads, in two kernels 23; clusters of 8 do not all find their SMs at once.
// The choice launched as a dependent of the scores: 28.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "fa_arrivals.cuh"
#include "fa_paged.cuh"
#include "fa_sm103.cuh"
#include "fa_store.cuh"
#include "ptx_sm103.cuh"

namespace fa {
namespace {

constexpr int kRows = 16;
constexpr int kGroup = 8;                  // pages of a warp's product
constexpr int kBins = 1024;
constexpr int kScoreThreads = 128;         // of a block that only scores
constexpr int score_ctas(bool flip) { return flip ? 4 : 3; }     // and such blocks on an SM (flip: 64 sequences of 1024 pages 40 us with 3)
constexpr int kJointThreads = 384;         // of a block that scores a share of the pages, one on an SM

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8)
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// hi + lo and hi - lo of four bounds each, as two pairs of fp16 (bytes 0, 1 and 2, 3): with their sign turned, the
// bytes are the low bits of 1152 + x, and all sums are whole numbers below 2048, exact.
__device__ __forceinline__ void sum_and_difference(uint32_t lo, uint32_t hi, uint32_t (&sum)[2], uint32_t (&diff)[2]) {
  const __half2 twice = __half2half2(__ushort_as_half(0x6880));            // 2304
  lo ^= 0x80808080u;
  hi ^= 0x80808080u;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t sel = e == 0 ? 0x4140 : 0x4342;
    const uint32_t x = __byte_perm(hi, 0x64646464u, sel), y = __byte_perm(lo, 0x64646464u, sel);
    const __half2 h = *reinterpret_cast<const __half2*>(&x), l = *reinterpret_cast<const __half2*>(&y);
    const __half2 d = __hsub2(h, l), s = __hadd2(__hsub2(h, twice), l);
    sum[e] = *reinterpret_cast<const uint32_t*>(&s);
    diff[e] = *reinterpret_cast<const uint32_t*>(&d);
  }
}

template <bool F16>
__device__ __forceinline__ float2 halves(uint32_t x) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  else return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// A slice's scores in the workspace
__host__ __device__ inline int64_t score_stride(int max_pages) { return ((int64_t)max_pages + 3) / 4 * 4; }

__device__ __forceinline__ int pages_of(const SelectArgs& a, int b) {
  if (new_tokens(a.q_lens, b, a.T) == 0) return 0;
  return (paged_len(a.cache, b, nullptr) + a.cache.page_size - 1) / a.cache.page_size;
}

// 16 rows of queries in whole numbers, fp16, converted once for a block, a row to a warp, by little code: a kernel this
// short runs from cold instruction caches, and a warp that converts all rows for itself takes 2 us for it.
template <int D>
struct Rows {
  static constexpr int kStride = D + 4;    // (8 bytes more: neighbouring rows in different banks)
  __align__(16) uint16_t q[kRows][kStride];
  float unit[kRows];                       // -1: no such row, or one that holds something not finite
};
template <int D, bool F16, int kThr, int kCount>
__device__ __forceinline__ void read_rows(const SelectArgs& a, int b, int hk, int row0, int count, Rows<D>& out) {
  constexpr int kOwn = D / 64;             // pairs of a lane
  const int lane = threadIdx.x % 32, G = a.H / a.Hkv, rows = G * a.T;
#pragma unroll 1
  for (int i = threadIdx.x / 32; i < kCount; i += kThr / 32) {
    const int r = row0 + i;
    const bool there = r < rows && r % a.T < count;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + (((int64_t)b * a.H + hk * G) * a.T + r) * D) +
                        lane * kOwn;
    float2 x[kOwn];
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      x[k] = halves<F16>(there ? __ldg(p + k) : 0u);
      amax = max(amax, max(__float_as_uint(x[k].x) & 0x7fffffffu, __float_as_uint(x[k].y) & 0x7fffffffu));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    const float u = power_scale<true>(amax), inv = 1.f / u;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const float y = rintf(x[k].x * inv), z = rintf(x[k].y * inv);
      reinterpret_cast<uint32_t*>(out.q[i])[lane * kOwn + k] = ptx::pack_f16(y, z);
    }
    if (lane == 0) out.unit[i] = there && amax < 0x7f800000u ? u : -1.f;
  }
}

// 16 rows as left operands, or 8 as right ones (kFlip): product 4 i + w takes the values [64 i + 16 (lane % 4) + 4 w, + 4) of
// a lane (k-columns 2 j, 2 j + 1, 2 j + 8, 2 j + 9 of lane j).
template <int D, bool F16, bool kFlip>
struct Queries {
  static constexpr int kHalves = kFlip ? 1 : 2;            // rows of a lane: lane / 4, and that and 8 more
  uint32_t q[D / 16][2 * kHalves];
  float unit[2];                           // of the rows of the lane's sums.  -1: no such row, or one that holds something not finite
  __device__ __forceinline__ void take(const Rows<D>& r) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int e = 0; e < kHalves; ++e) {
      const int row = lane / 4 + e * 8;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const uint2 x = *reinterpret_cast<const uint2*>(&r.q[row][j / 4 * 64 + lane % 4 * 16 + j % 4 * 4]);
        q[j][e] = x.x;
        q[j][e + kHalves] = x.y;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) unit[e] = r.unit[kFlip ? lane % 4 * 2 + e : lane / 4 + e * 8];
  }
  // ... or converted by the warp itself
  __device__ __forceinline__ void read(const SelectArgs& a, int b, int hk, int row0, int count) {
    const int lane = threadIdx.x % 32, G = a.H / a.Hkv, rows = G * a.T;
#pragma unroll
    for (int e = 0; e < kHalves; ++e) {
      const int r = row0 + lane / 4 + e * 8, t = r % a.T;
      const bool there = r < rows && t < count;
      const uint16_t* p = static_cast<const uint16_t*>(a.q) + (((int64_t)b * a.H + hk * G) * a.T + r) * D + lane % 4 * 16;
      float x[D / 4];
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint4 v = there ? __ldg(reinterpret_cast<const uint4*>(p + i * 64) + w) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = halves<F16>(u[k]);
            x[i * 16 + w * 8 + 2 * k] = f.x;
            x[i * 16 + w * 8 + 2 * k + 1] = f.y;
            amax = max(amax, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
          }
        }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const float u = power_scale<true>(amax), inv = 1.f / u;
      unit[e] = there && amax < 0x7f800000u ? u : -1.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          q[j][e + kHalves * k] = ptx::pack_f16(rintf(x[4 * j + 2 * k] * inv), rintf(x[4 * j + 2 * k + 1] * inv));
    }
    if constexpr (kFlip) {
      const float own = unit[0];
#pragma unroll
      for (int e = 0; e < 2; ++e) unit[e] = __shfl_sync(0xffffffffu, own, 4 * (lane % 4 * 2 + e));
    }
  }
};

// Whole numbers in the order of the scores; above all of them those of pages that are always chosen, below them of no page.
constexpr uint32_t kForcedKey = 0xffffffffu, kNanKey = 0xfffffffeu, kNoKey = 0u;
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return x != x ? kNanKey : (u >> 31) != 0u ? ~u : u | 0x80000000u;
}

// Scores of pages [p32, n) in steps of `step`, 32 at a time, for rows [row0, row0 + 16): put(page, score).
template <int D, bool F16, bool kFlip, typename Put>
__device__ __forceinline__ void score_pages(const SelectArgs& a, const Queries<D, F16, kFlip>& q, int b, int hk, int n, int p32,
                                            int step, Put&& put) {
  const int lane = threadIdx.x % 32;
  const int32_t* const table = a.cache.table + b * a.cache.table_stride;
  // 32 pages' places, one to a lane, read ahead
  auto places = [&](int p0) {
    const int p = p0 + lane;
    int page = p < n ? table[p] : -1;
    if (p < n && (unsigned)page >= (unsigned)a.cache.n_pages) {
      atomicExch(a.err, kDevBadOffsets);                 // reported, not followed
      page = -1;
    }
    return page;
  };
  int next = places(p32);
#pragma unroll 1
  for (; p32 < n; p32 += step) {
    const int lane_page = next;
    uint4 v[4][D / 32];
    float mine[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int page = __shfl_sync(0xffffffffu, lane_page, y * kGroup + lane / 4);
      const int64_t place = (int64_t)page * a.Hkv + hk;
      const uint4* const src = reinterpret_cast<const uint4*>(a.bounds + place * 2 * D) + lane % 4;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[y][i] = page >= 0 ? __ldg(src + i * 4) : make_uint4(0u, 0u, 0u, 0u);
      mine[y] = page >= 0 ? __ldg(a.bound_scales + place) : 0.f;
    }
    next = places(p32 + step);
    if constexpr (kFlip) {
      // two groups' pages are the rows of a product, the queries its columns
#pragma unroll
      for (int y = 0; y < 4; y += 2) {
        const int p = p32 + y * kGroup + lane / 4;
        if (p32 + y * kGroup >= n) break;
        float c[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t sum[4], diff[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4 lo = v[y + e][i], hi = v[y + e][D / 64 + i];
              const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
              uint32_t s2[2], d2[2];
              sum_and_difference(l[w], h[w], s2, d2);
              sum[e] = s2[0];
              sum[e + 2] = s2[1];
              diff[e] = d2[0];
              diff[e + 2] = d2[1];
            }
            const uint32_t q0 = q.q[4 * i + w][0], q1 = q.q[4 * i + w][1];
            mma(c, sum, q0, q1);
            mma(d, diff, q0 & 0x7fff7fffu, q1 & 0x7fff7fffu);
          }
        // the lane's sums: queries 2 (lane % 4) and the next, of pages lane / 4 and that and 8 more
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float best = fmaxf(q.unit[0] == -1.f ? -INFINITY : 0.5f * (c[2 * e] + d[2 * e]) * q.unit[0],
                             q.unit[1] == -1.f ? -INFINITY : 0.5f * (c[2 * e + 1] + d[2 * e + 1]) * q.unit[1]);
          best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
          best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
          if (lane % 4 == 0 && p + 8 * e < n) put(p + 8 * e, __fmul_rn(best, mine[y + e]));
        }
      }
    } else {
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int p0 = p32 + y * kGroup;
      if (p0 >= n) break;
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t lo[4] = {v[y][i].x, v[y][i].y, v[y][i].z, v[y][i].w};
        const uint4 up = v[y][D / 64 + i];
        const uint32_t hi[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t sum[2], diff[2], size[4];
          sum_and_difference(lo[w], hi[w], sum, diff);
          mma(c, q.q[4 * i + w], sum[0], sum[1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) size[k] = q.q[4 * i + w][k] & 0x7fff7fffu;
          mma(c, size, diff[0], diff[1]);
        }
      }
      // the lane's columns are pages 2 (lane % 4) and the next.  The scale is positive, so it may wait until
      // the largest is known; one that is NaN makes the score NaN.
      float best[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        best[e] = fmaxf(q.unit[0] == -1.f ? -INFINITY : 0.5f * c[e] * q.unit[0],
                        q.unit[1] == -1.f ? -INFINITY : 0.5f * c[2 + e] * q.unit[1]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) best[e] = fmaxf(best[e], __shfl_xor_sync(0xffffffffu, best[e], o));
        best[e] = __fmul_rn(best[e], __shfl_sync(0xffffffffu, mine[y], (2 * (lane % 4) + e) * 4));
      }
      if (lane < 4) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (p0 + 2 * lane + e < n) put(p0 + 2 * lane + e, best[e]);
      }
    }
    }
  }
}
__device__ __forceinline__ float larger_score(float x, float y) { return x != x || y != y ? x + y : fmaxf(x, y); }

// Scores by block `part` of the `parts` of a slice, neighbouring pages in different blocks: put(page, score, whether these are
// the first rows).
template <int D, bool F16, bool kFlip, int kThr, typename Put>
__device__ __forceinline__ void score_slice(const SelectArgs& a, int b, int hk, int n, int part, int parts, Put&& put) {
  __shared__ Rows<D> shared;
  const int rows = a.H / a.Hkv * a.T, count = new_tokens(a.q_lens, b, a.T);
  const int p0 = (threadIdx.x / 32 * parts + part) * 32, step = parts * kThr;
#pragma unroll 1
  for (int row0 = 0; row0 < rows; row0 += kRows) {
    if (row0 > 0) __syncthreads();                         // the rows before are read no more
    read_rows<D, F16, kThr, kFlip ? 8 : kRows>(a, b, hk, row0, count, shared);
    __syncthreads();
    if (p0 >= n) continue;
    Queries<D, F16, kFlip> q;
    q.take(shared);
    score_pages<D, F16, kFlip>(a, q, b, hk, n, p0, step, [&](int p, float x) { put(p, x, row0 == 0); });
  }
}

// Scores on all SMs: warp W of the grid takes slice W % slices, so that neighbours read neighbouring heads' bounds.
template <int D, bool F16, bool kFlip>
__global__ void __launch_bounds__(kScoreThreads, score_ctas(kFlip)) score_kernel(const SelectArgs a, const int slots) {
  const int warp = blockIdx.x * (kScoreThreads / 32) + threadIdx.x / 32, slices = a.B * a.Hkv;
  const int slice = warp % slices, slot = warp / slices;
  const int b = slice / a.Hkv, hk = slice % a.Hkv;
  const int n = pages_of(a, b);
  if (n <= a.picks || slot >= slots || slot * 32 >= n) return;   // all of them, or no page for this warp
  const int rows = a.H / a.Hkv * a.T, count = new_tokens(a.q_lens, b, a.T);
  float* const scores = a.scores + (int64_t)slice * score_stride(a.cache.max_pages);
  for (int row0 = 0; row0 < rows; row0 += kRows) {
    Queries<D, F16, kFlip> q;
    q.read(a, b, hk, row0, count);
    score_pages<D, F16, kFlip>(a, q, b, hk, n, slot * 32, slots * 32,
                        [&](int p, float x) { scores[p] = row0 > 0 ? larger_score(scores[p], x) : x; });
  }
}

// The choice among n pages, more than are wanted.  keys: the scores, a thread's own in fours (4 i to 4 i + 3 of i = its
// number + k kThr).  Little code, for the caches of instructions are cold: one page a lane wherever there is no more
// to it than a comparison.
template <int kThr>
__device__ __forceinline__ void choose(const SelectArgs& a, uint32_t* keys, int n, int32_t* out) {
  constexpr int kWarps = kThr / 32;
  constexpr int kPer = (kBins + kThr - 1) / kThr;        // bins of a thread
  __shared__ int hist[kPer * kThr];
  __shared__ uint32_t ends[2][kWarps];
  __shared__ int sums[2][kWarps];
  __shared__ int found[3];                               // bin, keys in it, keys wanted of it
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // pages that are always chosen, and the `want` highest of the others
  const int64_t always = (int64_t)a.first + a.last;
  int want = always < a.picks ? a.picks - (int)always : 0;
  // the scores' range
  uint32_t lo = 0xffffffffu, hi = 0u;
  uint4* const keys4 = reinterpret_cast<uint4*>(keys);
  const int n4 = (n + 3) / 4;
#pragma unroll 1
  for (int i = threadIdx.x; i < n4; i += kThr) {
    const uint4 v = keys4[i];
    uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = 4 * i + e;
      key[e] = order_of(__uint_as_float(key[e]));
      const bool own = p >= a.first && p < n - a.last;   // (n exceeds both)
      lo = own ? min(lo, key[e]) : lo;
      hi = own ? max(hi, key[e]) : hi;
      key[e] = own ? key[e] : p < n ? kForcedKey : kNoKey;
    }
    keys4[i] = make_uint4(key[0], key[1], key[2], key[3]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    ends[0][warp] = lo;
    ends[1][warp] = hi;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) hist[e * kThr + threadIdx.x] = 0;
  __syncthreads();
#pragma unroll 4
  for (int w = 0; w < kWarps; ++w) {
    lo = min(lo, ends[0][w]);
    hi = max(hi, ends[1][w]);
  }
  if (want == 0) {                                       // those that are always chosen alone
    lo = kForcedKey;
    hi = kNanKey;
  }
  // [lo, hi] holds the K-th largest key: `want` of the keys in it are chosen, and all above
#pragma unroll 1
  while (want > 0) {
    const int bits = 32 - __clz(hi - lo), shift = max(0, bits - 10);
#pragma unroll 1
    for (int i = threadIdx.x; i < n4; i += kThr) {
      const uint4 v = keys4[i];
      const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (key[e] - lo <= hi - lo) atomicAdd(&hist[(key[e] - lo) >> shift], 1);
    }
    __syncthreads();
    // thread t holds kPer bins, from the top
    int mine[kPer], sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      mine[e] = hist[kPer * kThr - 1 - kPer * threadIdx.x - e];
      sum += mine[e];
    }
    int up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    if (lane == 31) sums[0][warp] = up;
    __syncthreads();
    int before = up - sum;
#pragma unroll 4
    for (int w = 0; w < warp; ++w) before += sums[0][w];
    if (before < want && before + sum >= want) {
      bool open = true;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (open && before + mine[e] >= want) {
          found[0] = kPer * kThr - 1 - kPer * (int)threadIdx.x - e;
          found[1] = mine[e];
          found[2] = want - before;
          open = false;
        }
        before += mine[e];
      }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) hist[e * kThr + threadIdx.x] = 0;     // (all have read their bins)
    __syncthreads();
    const uint32_t at = lo + ((uint32_t)found[0] << shift);
    hi = min(hi, at + ((1u << shift) - 1u));
    lo = at;
    want = found[2];
    if (shift == 0 || found[1] == want) break;
  }
  // in page order, each warp a run of pages: keys above, and the first `want` of those in the range
  const int run = ((n + kWarps - 1) / kWarps + 31) / 32 * 32, begin = warp * run + lane, end = min(n, (warp + 1) * run);
  int above = 0, equal = 0;
#pragma unroll 4
  for (int i = begin; i < end; i += 32) {
    const uint32_t key = keys[i];
    above += key > hi ? 1 : 0;
    equal += key - lo <= hi - lo ? 1 : 0;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();                                       // sums is read no more
  if (lane == 0) {
    sums[0][warp] = above;
    sums[1][warp] = equal;
  }
  __syncthreads();
  above = equal = 0;
#pragma unroll 4
  for (int w = 0; w < warp; ++w) {
    above += sums[0][w];
    equal += sums[1][w];
  }
  const uint32_t lower = (1u << lane) - 1u;
#pragma unroll 1
  for (int i = begin; i - lane < end; i += 32) {
    const uint32_t key = i < end ? keys[i] : kNoKey;
    const bool up = key > hi, tie = key - lo <= hi - lo;
    const uint32_t ups = __ballot_sync(0xffffffffu, up), ties = __ballot_sync(0xffffffffu, tie);
    const int t = equal + __popc(ties & lower), at = above + __popc(ups & lower) + min(t, want);
    if ((up || (tie && t < want)) && at < a.picks) out[at] = i;          // (more that are always chosen: the first ones)
    above += __popc(ups);
    equal += __popc(ties);
  }
}

// Scores from the workspace to each thread's own keys.
template <int kThr>
__device__ __forceinline__ void take_scores(const float* scores, uint32_t* keys, int n) {
  const int n4 = (n + 3) / 4;
#pragma unroll 8
  for (int i = threadIdx.x; i < n4; i += kThr) reinterpret_cast<uint4*>(keys)[i] = __ldcg(reinterpret_cast<const uint4*>(scores) + i);
}

// kScored: score_kernel has been there.
template <int D, bool F16, bool kFlip, int kThr, bool kScored>
__global__ void __launch_bounds__(kThr, kThr == 128 ? 3 : 1) select_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];       // the pages' scores
  const int slice = blockIdx.x;
  const int b = slice / a.Hkv, hk = slice % a.Hkv;
  if (hk == 0 && threadIdx.x == 0) paged_len(a.cache, b, a.err);
  const int n = pages_of(a, b);
  int32_t* const out = a.pages + (int64_t)slice * a.picks;
  if (n <= a.picks) {                                    // all of them
    for (int i = threadIdx.x; i < a.picks; i += kThr) out[i] = i < n ? i : -1;
    return;
  }
  if constexpr (kScored) {
    take_scores<kThr>(a.scores + (int64_t)slice * score_stride(a.cache.max_pages), keys, n);
  } else {
    score_slice<D, F16, kFlip, kThr>(a, b, hk, n, 0, 1, [&](int p, float x, bool first) {
      keys[p] = __float_as_uint(first ? x : larger_score(__uint_as_float(keys[p]), x));
    });
    __syncthreads();
  }
  choose<kThr>(a, keys, n, out);
}

// Few slices: `parts` blocks score the pages of each, and the one that comes last chooses.
template <int D, bool F16, bool kFlip>
__global__ void __launch_bounds__(kJointThreads) joint_kernel(const SelectArgs a, const int parts) {
  extern __shared__ __align__(16) uint32_t keys[];       // the pages' scores
  __shared__ bool last;
  const int slices = a.B * a.Hkv, slice = blockIdx.x % slices, part = blockIdx.x / slices;
  const int b = slice / a.Hkv, hk = slice % a.Hkv;
  if (hk == 0 && part == 0 && threadIdx.x == 0) paged_len(a.cache, b, a.err);
  const int n = pages_of(a, b);
  int32_t* const out = a.pages + (int64_t)slice * a.picks;
  if (n <= a.picks) {                                    // all of them
    if (part == 0)
      for (int i = threadIdx.x; i < a.picks; i += kJointThreads) out[i] = i < n ? i : -1;
    return;
  }
  unsigned long long* const word = a.arrivals + slice;
  if (threadIdx.x == 0) open_count(word, a.call);
  float* const scores = a.scores + (int64_t)slice * score_stride(a.cache.max_pages);
  score_slice<D, F16, kFlip, kJointThreads>(a, b, hk, n, part, parts,
                                     [&](int p, float x, bool first) { scores[p] = first ? x : larger_score(scores[p], x); });
  __syncthreads();
  if (threadIdx.x == 0) {
    asm volatile("fence.acq_rel.gpu;" ::: "memory");     // releases what the whole block wrote before its barrier
    last = count_part(word, parts);
    if (last) asm volatile("fence.acq_rel.gpu;" ::: "memory");       // the scores, for the block after its barrier
  }
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) *word = 0ull;                    // for a captured call's next run under the same number
  take_scores<kJointThreads>(scores, keys, n);
  choose<kJointThreads>(a, keys, n, out);
}

template <int D, bool F16, bool kFlip, int kThr, bool kScored>
cudaError_t launch_one(const SelectArgs& a, cudaStream_t s) {
  auto kern = select_kernel<D, F16, kFlip, kThr, kScored>;
  static LaunchSetup setup;
  const int smem = a.cache.max_pages > a.picks ? (a.cache.max_pages + 3) / 4 * 16 : 0;
  const cudaError_t e = prepare_launch(setup, kern, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(a.B * a.Hkv), kThr, smem, s>>>(a);
  return cudaGetLastError();
}
// Few slices, of which each finds blocks on several SMs: they choose too.  (64 slices of up to 4000 pages: 24 us in two
// launches, 25.6 in one; 40 of up to 1250: 9.5 and 10.7.)
bool select_jointly(int slices, int sms) { return 4 * slices <= sms; }

template <int D, bool F16, bool kFlip>
cudaError_t launch_any(const SelectArgs& a, cudaStream_t s) {
  if (!select_scores_first(a.B, a.Hkv, a.cache.max_pages, a.picks))
    return a.cache.max_pages <= 512 ? launch_one<D, F16, kFlip, 128, false>(a, s) : launch_one<D, F16, kFlip, 256, false>(a, s);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int slices = a.B * a.Hkv;
  if (select_jointly(slices, sms)) {
    const int parts = std::min(sms / slices, (a.cache.max_pages + 31) / 32);
    static LaunchSetup setup;
    const int smem = (int)score_stride(a.cache.max_pages) * 4;
    if ((e = prepare_launch(setup, joint_kernel<D, F16, kFlip>, smem)) != cudaSuccess) return e;
    joint_kernel<D, F16, kFlip><<<slices * parts, kJointThreads, smem, s>>>(a, parts);
    return cudaGetLastError();
  }
  // warps of a slice: all take the same number of pages, as many warps as the SMs hold
  const int blocks = (a.cache.max_pages + 31) / 32;
  const int most = std::max(1, sms * score_ctas(kFlip) * (kScoreThreads / 32) / slices), each = (blocks + most - 1) / most;
  const int slots = (blocks + each - 1) / each;
  const int grid = (slots * slices + kScoreThreads / 32 - 1) / (kScoreThreads / 32);
  score_kernel<D, F16, kFlip><<<grid, kScoreThreads, 0, s>>>(a, slots);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // (the queries' type and size do not matter)
  return a.cache.max_pages <= 2048 ? launch_one<64, false, false, 256, true>(a, s) : launch_one<64, false, false, 1024, true>(a, s);
}

}  // namespace

// Whether the pages are scored on all SMs before the choice: where slices are not many times the SMs, each with more pages
// than a block scores while another launch begins (8 key heads of 4 rows, d = 128, 1024 pages: 32 sequences 28 us in one
// kernel and 22 in two, 64 sequences 54 and 36).
bool select_scores_first(int B, int Hkv, int max_pages, int picks) {
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess || sms <= 0) sms = 152;        // GB300's when no device can be asked
  return max_pages > picks && max_pages > 512 && (int64_t)B * Hkv <= 4 * (int64_t)sms;
}

size_t select_workspace(int B, int Hkv, int max_pages, size_t* arrivals) {
  *arrivals = (size_t)B * Hkv * score_stride(max_pages) * sizeof(float);
  return (*arrivals + (size_t)B * Hkv * sizeof(unsigned long long) + 255) / 256 * 256;
}

cudaError_t launch_select(const SelectArgs& a, fa_dtype dt, cudaStream_t s) {
  auto launch = [&](auto d, auto f16) {
    constexpr int D = decltype(d)::value;
    constexpr bool F16 = decltype(f16)::value;
    return a.H / a.Hkv * a.T <= 8 ? launch_any<D, F16, true>(a, s) : launch_any<D, F16, false>(a, s);
  };
  auto typed = [&](auto d) { return dt == FA_FP16 ? launch(d, std::true_type{}) : launch(d, std::false_type{}); };
  return a.d == 64 ? typed(std::integral_constant<int, 64>{}) : typed(std::integral_constant<int, 128>{});
}

}  // namespace fa
