// The choice of the pages that a sequence's next tokens attend to.
//
// For a query row q and a page whose keys lie between lo and hi in every one of the d values,
//     q . k <= sum_i max(q_i lo_i, q_i hi_i)
// for each of the page's keys.  With q in whole numbers of 2^f (8 bits, like lo and hi) the sum is
//     I = sum_i min(q_i, 0) lo_i + max(q_i, 0) hi_i,
// an inner product of 2 d whole numbers, below 2^24: exact in any order, so the choice does not depend on
// how the work is cut up.  A page's score is the largest over the rows of its key head's group of
// I * 2^f * (the bounds' scale); the first and the last pages, which are always chosen, and scores that are NaN
// stand above all others, and of equal ones the lower page is chosen.
//
// Scores.  A warp takes eight pages at a time: their bounds are the right operand of mma.sync's 8-bit
// whole-number form as they lie in memory, 16 rows' q the left one.  What bounds it: bytes, 2 d + 4 a page.
// Choice.  A block for each (sequence, key head) finds the K-th largest score by its bits, eight at a time,
// and lists the pages at or above it in their order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "fa_paged.cuh"
#include "fa_sm103.cuh"
#include "fa_store.cuh"
#include "ptx_sm103.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;
constexpr int kGroup = 8;                  // pages of a warp's product
constexpr int kPickThreads = 512;

// c (16 x 8, int32) += a (16 x 32) b (32 x 8)
__device__ __forceinline__ void mma_s8(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool F16>
__device__ __forceinline__ float2 halves(uint32_t x) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  else return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

__device__ __forceinline__ int pages_of(const SelectArgs& a, int b) {
  if (new_tokens(a.q_lens, b, a.T) == 0) return 0;
  return (paged_len(a.cache, b, nullptr) + a.cache.page_size - 1) / a.cache.page_size;
}

// 16 rows of queries as the left operand: products 4 j to 4 j + 3 of a lane's 64 bytes [64 i + 16 (lane % 4), + 16)
// of a page's lower (then upper) bounds, and what their whole numbers count.
template <int D, bool F16>
struct Queries {
  uint32_t low[D / 32][4], high[D / 32][4];
  float unit[2];                           // -1: no such row
  __device__ __forceinline__ void read(const SelectArgs& a, int b, int hk, int row0, int count) {
    const int lane = threadIdx.x % 32, G = a.H / a.Hkv, rows = G * a.T;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + lane / 4 + e * 8, t = r % a.T;
      const bool there = r < rows && t < count;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + (((int64_t)b * a.H + hk * G) * a.T + r) * D + lane % 4 * 16;
      float x[D / 4];
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint4 v = there ? __ldg(reinterpret_cast<const uint4*>(q + i * 64) + w) : make_uint4(0u, 0u, 0u, 0u);
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
      unit[e] = !there ? -1.f : amax < 0x7f800000u ? u : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int j = 0; j < D / 32; ++j)     // two products of 8 bytes of a lane's 16
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          int c[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) c[y] = __float2int_rn(x[8 * j + 4 * k + y] * inv);
          low[j][e + 2 * k] = pack_s8(min(c[0], 0), min(c[1], 0), min(c[2], 0), min(c[3], 0));
          high[j][e + 2 * k] = pack_s8(max(c[0], 0), max(c[1], 0), max(c[2], 0), max(c[3], 0));
        }
    }
  }
};

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps) score_kernel(const SelectArgs a, const int chunks) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int b = slice / a.Hkv, hk = slice % a.Hkv;
  const int n = pages_of(a, b);
  if (n <= a.picks) return;                             // all of them
  const int rows = a.H / a.Hkv * a.T, count = new_tokens(a.q_lens, b, a.T);
  const int32_t* const table = a.cache.table + b * a.cache.table_stride;
  float* const scores = a.scores + (int64_t)slice * a.cache.max_pages;
  const int step = chunks * kWarps * kGroup;
  for (int row0 = 0; row0 < rows; row0 += kRows) {
    Queries<D, F16> q;
    q.read(a, b, hk, row0, count);
    for (int p0 = (chunk * kWarps + warp) * kGroup; p0 < n; p0 += step) {
      const int p = p0 + lane / 4;
      int page = p < n ? table[p] : -1;
      if (p < n && (unsigned)page >= (unsigned)a.cache.n_pages) {
        atomicExch(a.err, kDevBadOffsets);              // reported, not followed
        page = -1;
      }
      const int64_t place = (int64_t)page * a.Hkv + hk;
      uint4 v[D / 32];
      const uint4* const src = reinterpret_cast<const uint4*>(a.bounds + place * 2 * D) + lane % 4;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[i] = page >= 0 ? __ldg(src + i * 4) : make_uint4(0u, 0u, 0u, 0u);
      const float mine = page >= 0 ? __ldg(a.bound_scales + place) : 0.f;
      int c[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        mma_s8(c, q.low[2 * i], v[i].x, v[i].y);
        mma_s8(c, q.low[2 * i + 1], v[i].z, v[i].w);
        mma_s8(c, q.high[2 * i], v[D / 64 + i].x, v[D / 64 + i].y);
        mma_s8(c, q.high[2 * i + 1], v[D / 64 + i].z, v[D / 64 + i].w);
      }
      // the lane's columns are pages 2 (lane % 4) and the next; -inf: no such row
      float best[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float s = __shfl_sync(0xffffffffu, mine, (2 * (lane % 4) + e) * 4);
        best[e] = -INFINITY;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float x = __fmul_rn(__fmul_rn((float)c[2 * w + e], q.unit[w]), s);
          // NaN: of the page, in every row; a row that is NaN itself has no say next to others
          best[e] = q.unit[w] == -1.f ? best[e] : best[e] == -INFINITY ? x : fmaxf(best[e], x);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          const float other = __shfl_xor_sync(0xffffffffu, best[e], o);
          best[e] = best[e] == -INFINITY ? other : other == -INFINITY ? best[e] : fmaxf(best[e], other);
        }
      }
      if (lane < 4) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = p0 + 2 * lane + e;
          if (at >= n) break;
          if (row0 > 0) {
            const float before = scores[at];
            best[e] = best[e] == -INFINITY ? before : before == -INFINITY ? best[e] : fmaxf(best[e], before);
          }
          scores[at] = best[e];
        }
      }
    }
  }
}

// Whole numbers in the order of the scores
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return x != x ? 0xffffffffu : (u >> 31) != 0u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[256];
  __shared__ int sums[2][kPickThreads / 32];
  __shared__ uint32_t digit_found;
  __shared__ int want_left;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.x / a.Hkv;
  if (blockIdx.x % a.Hkv == 0 && threadIdx.x == 0) paged_len(a.cache, b, a.err);
  const int n = pages_of(a, b);
  int32_t* const out = a.pages + (int64_t)blockIdx.x * a.picks;
  if (n <= a.picks) {
    for (int i = threadIdx.x; i < a.picks; i += kPickThreads) out[i] = i < n ? i : -1;
    return;
  }
  const float* const scores = a.scores + (int64_t)blockIdx.x * a.cache.max_pages;
  for (int i = threadIdx.x; i < n; i += kPickThreads)
    keys[i] = i < a.first || i >= n - a.last ? 0xffffffffu : order_of(__ldcg(scores + i));
  // the K-th largest key: its bits from the top, and how many of the keys equal to it are chosen
  uint32_t prefix = 0, mask = 0;
  int want = a.picks;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kPickThreads) hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPickThreads)
      if ((keys[i] & mask) == prefix) atomicAdd(&hist[(keys[i] >> shift) & 255u], 1);
    __syncthreads();
    if (warp == 0) {
      // lane i holds digits 255 - 8 i down to 248 - 8 i
      int mine[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mine[e] = hist[255 - 8 * lane - e];
        sum += mine[e];
      }
      int up = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
      }
      int before = up - sum;
      if (before < want && up >= want) {
        bool open = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (open && before + mine[e] >= want) {
            digit_found = 255 - 8 * lane - e;
            want_left = want - before;
            open = false;
          }
          before += mine[e];
        }
      }
    }
    __syncthreads();
    prefix |= digit_found << shift;
    mask |= 255u << shift;
    want = want_left;
    __syncthreads();
  }
  // in page order: keys above, and the first `want` of those equal
  int above = 0, equal = 0;
  for (int i0 = 0; i0 < n; i0 += kPickThreads) {
    const int i = i0 + threadIdx.x;
    const uint32_t key = i < n ? keys[i] : 0u;
    const bool up = i < n && key > prefix, tie = i < n && key == prefix;
    const uint32_t ups = __ballot_sync(0xffffffffu, up), ties = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) {
      sums[0][warp] = __popc(ups);
      sums[1][warp] = __popc(ties);
    }
    __syncthreads();
    int u = above, t = equal;
    for (int w = 0; w < kPickThreads / 32; ++w) {
      if (w < warp) {
        u += sums[0][w];
        t += sums[1][w];
      }
      above += sums[0][w];
      equal += sums[1][w];
    }
    u += __popc(ups & ((1u << lane) - 1u));
    t += __popc(ties & ((1u << lane) - 1u));
    if (up) out[u + min(t, want)] = i;
    else if (tie && t < want) out[u + t] = i;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, fa_dtype dt, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (a.cache.max_pages > a.picks) {
    const int64_t slices = (int64_t)a.B * a.Hkv;
    const int chunks = (a.cache.max_pages + kWarps * kGroup - 1) / (kWarps * kGroup);
    int64_t want = (16 * (int64_t)sms + slices - 1) / slices;
    if (want > chunks) want = chunks;
    const unsigned grid = (unsigned)(want * slices);
    if (a.d == 64) {
      if (dt == FA_FP16) score_kernel<64, true><<<grid, 32 * kWarps, 0, s>>>(a, (int)want);
      else score_kernel<64, false><<<grid, 32 * kWarps, 0, s>>>(a, (int)want);
    } else {
      if (dt == FA_FP16) score_kernel<128, true><<<grid, 32 * kWarps, 0, s>>>(a, (int)want);
      else score_kernel<128, false><<<grid, 32 * kWarps, 0, s>>>(a, (int)want);
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  static LaunchSetup setup;
  const int smem = a.cache.max_pages > a.picks ? a.cache.max_pages * 4 : 0;
  if ((e = prepare_launch(setup, pick_kernel, smem)) != cudaSuccess) return e;
  pick_kernel<<<(unsigned)(a.B * a.Hkv), kPickThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
