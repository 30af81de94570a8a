// Rotary positions: the rotation of query and key heads, its gradient, and the write of new
// tokens into a paged cache that rotates their keys (and queries) on the way.
//
// Pair i of a head, (a, b), at position t becomes m * (a cos w - b sin w, a sin w + b cos w),
// w = t * inv_freq[i].  The map is linear and, apart from m, orthogonal: its gradient is the
// rotation by -w with the same factor m.
//
// What bounds it: bytes.  Every value is read once and written once, with six flops a pair.
//
// The angle.  t * inv_freq in 32 bits loses the angle of far positions (at t = 10^6 the product
// is off by up to 0.03 rad), and 64-bit floating-point products run at a fiftieth of the 32-bit
// rate here.  Only the fraction of a turn matters, so each thread turns its frequencies once into
// 64-bit fixed point, F = inv_freq / (2 pi) * 2^64 mod 2^64 (the long product with the digits of
// 1 / (2 pi) is Payne and Hanek's reduction); the product t * F then wraps modulo one turn by itself,
// and its upper 32 bits are the angle to 2^-32 turns.  F is exact to 2^-63 turns a position, so a
// position of 2^31 still has an angle good to 2^-32 turns.  The sine takes it in fp32, whose 24 bits
// move it by up to 2^-26 turns (pi 2^-25), as much as the rounding of the sine itself: 16-bit
// results do not see that, fp32 ones have 1.3 times the error of sines taken in 64 bits.
//
// Layout.  A thread holds one unit of a token's heads: 8 pairs, the 16 values they occupy (two
// 16-byte loads in either pairing of a 16-bit type), and walks over heads with the sines and
// cosines it computed once.  Neighbouring threads take neighbouring units, then tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fa_paged.cuh"
#include "fa_rotate.cuh"
#include "fa_sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;                  // heads whose values a thread has in flight together

template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, const int heads_per_block) {
  const int units = a.d / kUnit;
  const int u = threadIdx.x % units;
  const Unit t = unit_of(u, a.rot);
  uint64_t frac[8];
  if (t.turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) frac[i] = turn_fraction(a.rot.inv_freq[8 * u + i]);
  }
  const int h0 = blockIdx.y * heads_per_block, h1 = min(a.H, h0 + heads_per_block);
  const int64_t tokens = (int64_t)a.B * a.N;
  const int per_block = kThreads / units;
  for (int64_t m = (int64_t)blockIdx.x * per_block + threadIdx.x / units; m < tokens;
       m += (int64_t)gridDim.x * per_block) {
    const int64_t b = m / a.N, n = m % a.N;
    const T* x = static_cast<const T*>(a.x) + b * a.xs.b + n * a.xs.n + h0 * a.xs.h;
    T* y = static_cast<T*>(a.y) + b * a.ys.b + n * a.ys.n + h0 * a.ys.h;
    // kBatch heads at a time: their reads are all in flight before the first is used, the first
    // ones' while the sines are computed
    Raw8<T> lo[kBatch], hi[kBatch];
    auto read = [&](int h) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < h1) {
          lo[i] = load8(x + i * a.xs.h + t.lo);
          hi[i] = load8(x + i * a.xs.h + t.hi);
        }
      x += kBatch * a.xs.h;
    };
    read(h0);
    float c[8], s[8];
    if (t.turns) angles(frac, a.positions[b * a.pos_stride + n], a.rot, c, s);
    for (int h = h0; h < h1; h += kBatch) {
      if (h > h0) read(h);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < h1) {
          if (t.turns) turn_raw(lo[i], hi[i], a.rot.interleaved, c, s);
          store8(y + i * a.ys.h + t.lo, lo[i]);
          store8(y + i * a.ys.h + t.hi, hi[i]);
        }
      y += kBatch * a.ys.h;
    }
  }
}

// New tokens of every sequence.  Heads are numbered through: H query heads (when there are
// queries), Hkv key heads, Hkv value heads; a block takes a range of them.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a, const int heads_per_block) {
  const int units = a.d / kUnit;
  const int u = threadIdx.x % units;
  const Unit t = unit_of(u, a.rot);
  const int Hq = a.q != nullptr ? a.H : 0;
  const int h0 = blockIdx.y * heads_per_block, h1 = min(Hq + 2 * a.Hkv, h0 + heads_per_block);
  const bool turns = t.turns && h0 < Hq + a.Hkv;
  uint64_t frac[8];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) frac[i] = turn_fraction(a.rot.inv_freq[8 * u + i]);
  }
  const int64_t tokens = (int64_t)a.B * a.T;
  const int per_block = kThreads / units;
  for (int64_t m = (int64_t)blockIdx.x * per_block + threadIdx.x / units; m < tokens;
       m += (int64_t)gridDim.x * per_block) {
    const int b = (int)(m / a.T), n = (int)(m % a.T);
    // the token's place in its sequence; padding of a ragged batch has none
    const int count = new_tokens(a.q_lens, b, a.T);
    const int pos = paged_len(a.cache, b, a.err) - count + n;
    const bool there = n < count && pos >= 0;
    int page = -1, slot = 0;
    if (there) {
      page = a.cache.table[b * a.cache.table_stride + pos / a.cache.page_size];
      slot = pos % a.cache.page_size;
      if ((unsigned)page >= (unsigned)a.cache.n_pages) {      // reported, not followed
        atomicExch(a.err, kDevBadOffsets);
        page = -1;
      }
    }
    const int64_t row = (int64_t)page * a.cache.page_stride + (int64_t)slot * a.cache.token_stride;
    float c[8], s[8];
    if (turns && there) angles(frac, pos, a.rot, c, s);
    for (int h = h0; h < h1; h += kBatch) {
      Raw8<T> lo[kBatch], hi[kBatch];
      T* to[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool is_q = h + i < Hq, is_k = !is_q && h + i < Hq + a.Hkv;
        const int g = is_q ? h + i : is_k ? h + i - Hq : h + i - Hq - a.Hkv;
        const Strides st = is_q ? a.qs : is_k ? a.ks : a.vs;
        to[i] = nullptr;
        if (h + i >= h1 || (!is_q && page < 0)) continue;
        to[i] = is_q ? static_cast<T*>(a.q_out) + (((int64_t)b * a.H + g) * a.T + n) * a.d
                     : static_cast<T*>(is_k ? a.cache.k : a.cache.v) + row + g * a.cache.head_stride;
        lo[i] = hi[i] = Raw8<T>{};                    // queries that do not exist: zero
        if (there) {
          const T* x = static_cast<const T*>(is_q ? a.q : is_k ? a.k : a.v) + b * st.b + g * st.h + n * st.n;
          lo[i] = load8(x + t.lo);
          hi[i] = load8(x + t.hi);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (to[i] == nullptr) continue;
        // values are copied, and so is the part of a head that is not rotated
        if (t.turns && there && h + i < Hq + a.Hkv) turn_raw(lo[i], hi[i], a.rot.interleaved, c, s);
        store8(to[i] + t.lo, lo[i]);
        store8(to[i] + t.hi, hi[i]);
      }
    }
  }
}

// Heads a block walks over.  More of them share one computation of the sines; fewer give small
// calls more blocks: halved until there are eight blocks of 128 threads per SM, about two waves.
// (Cache write of 4 ragged prompts of 4096 tokens, 48 heads: 63 us; with two or four per SM 70, with 32
// per SM 84.)
int heads_per_block(int64_t token_blocks, int heads, int sms) {
  const int least = (heads + 65534) / 65535;          // a grid's second axis
  int per = heads;
  while (per > least && token_blocks * ((heads + per - 1) / per) < 8 * sms) per = std::max(least, (per + 1) / 2);
  return per;
}

template <typename T>
cudaError_t rotary(const RotaryArgs& a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int per_block = kThreads / (a.d / kUnit);
  const int64_t blocks = ((int64_t)a.B * a.N + per_block - 1) / per_block;
  const int hp = heads_per_block(blocks, a.H, sms);
  const int64_t cap = 1 << 20;                      // the rest by the kernel's loop over tokens
  rotary_kernel<T><<<dim3((unsigned)(blocks < cap ? blocks : cap), (a.H + hp - 1) / hp), kThreads, 0, s>>>(a, hp);
  return cudaGetLastError();
}

template <typename T>
cudaError_t append(const AppendArgs& a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int per_block = kThreads / (a.d / kUnit);
  const int64_t blocks = ((int64_t)a.B * a.T + per_block - 1) / per_block;
  const int heads = (a.q != nullptr ? a.H : 0) + 2 * a.Hkv;
  const int hp = heads_per_block(blocks, heads, sms);
  const int64_t cap = 1 << 20;
  append_kernel<T><<<dim3((unsigned)(blocks < cap ? blocks : cap), (heads + hp - 1) / hp), kThreads, 0, s>>>(a, hp);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_FP32) return rotary<float>(a, s);
  return dt == FA_FP16 ? rotary<__half>(a, s) : rotary<__nv_bfloat16>(a, s);
}

cudaError_t launch_append(const AppendArgs& a, fa_dtype dt, cudaStream_t s) {
  return dt == FA_FP16 ? append<__half>(a, s) : append<__nv_bfloat16>(a, s);
}

}  // namespace fa
