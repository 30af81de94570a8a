// Arguments and launchers of the rotary, cache-write and paged-attention kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_internal.cuh"

namespace fa {

// The error word kernels write to in the current context (defined in fa_api.cu).
fa_status device_error_word(int** out);

// Rotation of pairs by position (see fa_rotary).
struct Rotation {
  const double* inv_freq;    // [rot / 2] radians per position; null with rot = 0
  int rot;                   // leading values of each head that are rotated (a multiple of 16)
  int interleaved;           // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
  float mscale;              // multiplies the rotated values
  float sign;                // -1 turns backwards (the gradient)
};

struct Strides {             // elements between batches, heads and tokens; values of a head adjoin
  int64_t b, h, n;
};

struct RotaryArgs {
  const void* x;
  void* y;
  Strides xs, ys;
  int B, H, N, d;
  const int32_t* positions;
  int64_t pos_stride;        // elements between batches; 0: one list for all
  Rotation rot;
};

// Pages of keys and values (see fa_paged_cache), and where each sequence's tokens are.
struct PagedCache {
  void* k;
  void* v;
  int64_t page_stride, head_stride, token_stride;
  int n_pages, page_size;
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
  const int32_t* kv_lens;
};

struct AppendArgs {
  PagedCache cache;
  const void* q;             // null: no queries
  const void* k;
  const void* v;
  void* q_out;               // [B, H, T, d]
  Strides qs, ks, vs;
  int B, H, Hkv, T, d;
  const int32_t* q_lens;     // null: T new tokens each
  Rotation rot;
  int* err;
};

struct PagedArgs {
  PagedCache cache;
  const void* q;             // [B, H, T, d]
  void* o;
  float* lse;
  int B, H, Hkv, T, d;
  const int32_t* q_lens;
  float scale;
  ScoreArgs score;           // cap and slopes; no prefix
  // page_size / 16, and 2^36 / that rounded up
  uint32_t page_parts;
  uint64_t parts_magic;
  // arrivals [2 * ctas]: the words that announce the parts; fp32 partial results, two parts per CTA:
  // o_part [2 * ctas][16][d] un-normalised, ml_part
  // [2 * ctas][16] = {log2-domain maximum, normaliser}
  unsigned long long* arrivals;
  unsigned long long call;   // the call's number
  float* o_part;
  float2* ml_part;
  int ctas;
  int* err;
};

// A sequence's valid keys and its new tokens.  A length beyond the table's pages breaks the
// contract: the sequence then has no keys (the caller's error word tells).
__host__ __device__ inline int paged_capacity(const PagedCache& c) {
  const int64_t cap = (int64_t)c.max_pages * c.page_size;
  return cap > 0x7ffffff0 ? 0x7ffffff0 : (int)cap;
}
__device__ __forceinline__ int paged_len(const PagedCache& c, int b, int* err) {
  const int n = c.kv_lens[b];
  if (n > paged_capacity(c)) {
    if (err != nullptr) atomicExch(err, kDevBadOffsets);
    return 0;
  }
  return n < 0 ? 0 : n;
}
__device__ __forceinline__ int new_tokens(const int32_t* q_lens, int b, int T) {
  if (q_lens == nullptr) return T;
  const int n = q_lens[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

cudaError_t launch_rotary(const RotaryArgs& a, fa_dtype dt, cudaStream_t s);
cudaError_t launch_append(const AppendArgs& a, fa_dtype dt, cudaStream_t s);

// CTAs of a paged attention call, and the bytes of its partial results.
// Pages of up to 4096 tokens: part * (rounding of the reciprocal) stays below 2^36 for any part of
// a sequence of 2^31 tokens, which the kernel's division by multiplication needs.
constexpr int kMaxPageSize = 4096;
int paged_ctas();
unsigned long long paged_call_number();
bool paged_shares(int B, int Hkv, int rows, int capacity, int ctas);
bool paged_counts(int B, int Hkv, int rows, int capacity);
struct PagedWorkspace {
  size_t ml, o, total;       // byte offsets; arrivals at 0
};
PagedWorkspace paged_workspace(int ctas, int d);
cudaError_t launch_paged(const PagedArgs& a, fa_dtype dt, cudaStream_t s);

}  // namespace fa
