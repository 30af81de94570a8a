// C-ABI layer of the rotary, cache-write and paged-attention calls: argument checks and launches.
// See include/fa.h for the contract.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "fa_paged.cuh"
#include "fa_score.cuh"
#include "fa_sm103.cuh"

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Sizes every call here shares.  Tokens and heads stay below 2^31 in all, so that a grid and the
// row numbers fit.
fa_status check_sizes(int B, int H, int Hkv, int N, int d) {
  if (B < 0 || H < 0 || N < 0 || Hkv < 0 || (H > 0 && Hkv == 0)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (H > 65535 || Hkv > 65535 || B > 65535) return FA_ERR_UNSUPPORTED;
  if (H > 0 && (Hkv > H || H % Hkv != 0)) return FA_ERR_UNSUPPORTED;
  if ((int64_t)B * (H > 0 ? H : 1) * N > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// 16-byte accesses: every stride that is stepped over keeps the alignment.
bool strides_ok(const int64_t* s, int B, int H, int N, int size) {
  if (s == nullptr) return false;
  const int64_t unit = 16 / size;
  return (B <= 1 || s[0] % unit == 0) && (H <= 1 || s[1] % unit == 0) && (N <= 1 || s[2] % unit == 0);
}

// Whether no two elements of a written tensor share memory: taken by growing stride, every axis steps
// over all that the ones before it span.
bool apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int d) {
  struct Axis { int64_t n, s; } x[3] = {{n0, s0}, {n1, s1}, {n2, s2}};
  std::sort(x, x + 3, [](const Axis& a, const Axis& b) { return a.s < b.s; });
  int64_t span = d;
  for (const Axis& a : x) {
    if (a.n <= 1) continue;
    if (a.s < span) return false;
    span += (a.n - 1) * a.s;
  }
  return true;
}

fa::Strides strides(const int64_t* s) { return fa::Strides{s[0], s[1], s[2]}; }

fa_status check_rotation(const double* inv_freq, int rotary_dim, float mscale, int d) {
  if (rotary_dim < 0) return FA_ERR_INVALID_ARG;
  if (rotary_dim > d || rotary_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (rotary_dim > 0 && (inv_freq == nullptr || !aligned(inv_freq, 8) || !isfinite(mscale))) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_cache(const fa_paged_cache* c, int Hkv) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  if (c->n_pages < 0 || c->max_pages < 0 || c->page_size <= 0) return FA_ERR_INVALID_ARG;
  if (c->page_size % 16 != 0 || c->page_size > fa::kMaxPageSize) return FA_ERR_UNSUPPORTED;
  if (!c->k_cache || !c->v_cache || (!c->block_table && c->max_pages > 0) || !c->kv_lens) return FA_ERR_INVALID_ARG;
  if (!aligned(c->k_cache, 16) || !aligned(c->v_cache, 16) || !aligned(c->block_table, 4) || !aligned(c->kv_lens, 4))
    return FA_ERR_INVALID_ARG;
  if (c->token_stride % 8 != 0 || (c->n_pages > 1 && c->page_stride % 8 != 0) || (Hkv > 1 && c->head_stride % 8 != 0))
    return FA_ERR_INVALID_ARG;
  if (c->table_stride < c->max_pages) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa::PagedCache cache_args(const fa_paged_cache* c) {
  fa::PagedCache p{};
  p.k = c->k_cache;
  p.v = c->v_cache;
  p.page_stride = c->page_stride;
  p.head_stride = c->head_stride;
  p.token_stride = c->token_stride;
  p.n_pages = c->n_pages;
  p.page_size = c->page_size;
  p.table = c->block_table;
  p.table_stride = c->table_stride;
  p.max_pages = c->max_pages;
  p.kv_lens = c->kv_lens;
  return p;
}

fa_status rotary_impl(const void* x, const int64_t* xs, void* y, const int64_t* ys, int B, int H, int N, int d,
                      const int32_t* positions, int64_t position_stride, const double* inv_freq,
                      int rotary_dim, int interleaved, float mscale, float sign, fa_dtype dtype, void* stream) {
  fa_status st = check_sizes(B, H, H, N, d);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP16 && dtype != FA_FP32) return FA_ERR_UNSUPPORTED;
  st = check_rotation(inv_freq, rotary_dim, mscale, d);
  if (st != FA_OK) return st;
  if (B == 0 || H == 0 || N == 0) return FA_OK;
  const int size = dtype == FA_FP32 ? 4 : 2;
  if (!x || !y || !positions || !aligned(x, 16) || !aligned(y, 16) || !aligned(positions, 4)) return FA_ERR_INVALID_ARG;
  if (!strides_ok(xs, B, H, N, size) || !strides_ok(ys, B, H, N, size) || position_stride < 0) return FA_ERR_INVALID_ARG;
  if (!apart(B, ys[0], H, ys[1], N, ys[2], d)) return FA_ERR_INVALID_ARG;
  fa::RotaryArgs a{};
  a.x = x;
  a.y = y;
  a.xs = strides(xs);
  a.ys = strides(ys);
  a.B = B; a.H = H; a.N = N; a.d = d;
  a.positions = positions;
  a.pos_stride = position_stride;
  a.rot = fa::Rotation{inv_freq, rotary_dim, interleaved != 0, mscale, sign};
  return fa::launch_rotary(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

fa_status fa_rotary(const void* x, const int64_t x_strides[3], void* y, const int64_t y_strides[3], int B, int H,
                    int N, int d, const int32_t* positions, int64_t position_stride, const double* inv_freq,
                    int rotary_dim, int interleaved, float mscale, fa_dtype dtype, void* stream) {
  return rotary_impl(x, x_strides, y, y_strides, B, H, N, d, positions, position_stride, inv_freq, rotary_dim,
                     interleaved, mscale, 1.f, dtype, stream);
}

fa_status fa_rotary_backward(const void* dy, const int64_t dy_strides[3], void* dx, const int64_t dx_strides[3],
                             int B, int H, int N, int d, const int32_t* positions, int64_t position_stride,
                             const double* inv_freq, int rotary_dim, int interleaved, float mscale,
                             fa_dtype dtype, void* stream) {
  return rotary_impl(dy, dy_strides, dx, dx_strides, B, H, N, d, positions, position_stride, inv_freq,
                     rotary_dim, interleaved, mscale, -1.f, dtype, stream);
}

fa_status fa_append_paged(const fa_paged_cache* cache, const void* k, const int64_t k_strides[3], const void* v,
                          const int64_t v_strides[3], const void* q, const int64_t q_strides[3], void* q_out,
                          int B, int H, int Hkv, int T, int d, const int32_t* q_lens, const double* inv_freq,
                          int rotary_dim, int interleaved, float mscale, fa_dtype dtype, void* stream) {
  // without queries the number of their heads does not matter; with some there have to be heads
  if (H < 0 || (q != nullptr && H == 0 && Hkv > 0)) return FA_ERR_INVALID_ARG;
  if (q == nullptr) H = Hkv;
  fa_status st = check_sizes(B, H, Hkv, T, d);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  st = check_rotation(inv_freq, rotary_dim, mscale, d);
  if (st != FA_OK) return st;
  if (B == 0 || Hkv == 0 || T == 0) return FA_OK;
  st = check_cache(cache, Hkv);
  if (st != FA_OK) return st;
  // the pages are written
  if (cache->k_cache == cache->v_cache || !apart(cache->n_pages, cache->page_stride, Hkv, cache->head_stride,
                                                 cache->page_size, cache->token_stride, d))
    return FA_ERR_INVALID_ARG;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_lens, 4)) return FA_ERR_INVALID_ARG;
  if (!strides_ok(k_strides, B, Hkv, T, 2) || !strides_ok(v_strides, B, Hkv, T, 2)) return FA_ERR_INVALID_ARG;
  if (q != nullptr && (!q_out || !aligned(q, 16) || !aligned(q_out, 16) || !strides_ok(q_strides, B, H, T, 2)))
    return FA_ERR_INVALID_ARG;
  fa::AppendArgs a{};
  a.cache = cache_args(cache);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  if (q != nullptr) a.qs = strides(q_strides);
  a.ks = strides(k_strides);
  a.vs = strides(v_strides);
  a.B = B; a.H = H; a.Hkv = Hkv; a.T = T; a.d = d;
  a.q_lens = q_lens;
  a.rot = fa::Rotation{inv_freq, rotary_dim, interleaved != 0, mscale, 1.f};
  if (fa::device_error_word(&a.err) != FA_OK) return FA_ERR_CUDA;
  return fa::launch_append(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_forward_paged_workspace_size(int B, int H, int Hkv, int T, int d, int max_keys) {
  if (check_sizes(B, H, Hkv, T, d) != FA_OK || B == 0 || H == 0 || T == 0 || max_keys <= 0) return 0;
  const int ctas = fa::paged_ctas();
  return fa::paged_shares(B, Hkv, H / Hkv * T, max_keys, ctas) ? fa::paged_workspace(ctas, d).total : 0;
}

fa_status fa_forward_paged(const void* q, const fa_paged_cache* cache, void* o, float* lse, int B, int H, int Hkv,
                           int T, int d, float scale, const int32_t* q_lens, const fa_score_mod* score,
                           fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_sizes(B, H, Hkv, T, d);
  if (st != FA_OK) return st;
  if (!isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (score != nullptr) {
    if (!isfinite(score->softcap) || score->softcap < 0.f || !aligned(score->alibi_slopes, 4)) return FA_ERR_INVALID_ARG;
    if (score->prefix_lens != nullptr) return FA_ERR_UNSUPPORTED;
  }
  fa::ScoreArgs mods;
  if (!fa::make_score(score, scale, &mods)) return FA_ERR_UNSUPPORTED;
  if (B == 0 || H == 0 || T == 0) return FA_OK;
  st = check_cache(cache, Hkv);
  if (st != FA_OK) return st;
  if (!q || !o || !lse || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(q_lens, 4))
    return FA_ERR_INVALID_ARG;
  fa::PagedArgs a{};
  a.cache = cache_args(cache);
  const size_t need = fa_forward_paged_workspace_size(B, H, Hkv, T, d, fa::paged_capacity(a.cache));
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.B = B; a.H = H; a.Hkv = Hkv; a.T = T; a.d = d;
  a.q_lens = q_lens;
  a.scale = scale;
  a.score = mods;
  if (!fa::paged_counts(B, Hkv, H / Hkv * T, fa::paged_capacity(a.cache))) return FA_ERR_UNSUPPORTED;
  a.page_parts = cache->page_size / 16;
  a.parts_magic = ((uint64_t(1) << 36) + a.page_parts - 1) / a.page_parts;
  a.ctas = fa::paged_ctas();
  const fa::PagedWorkspace w = fa::paged_workspace(a.ctas, d);
  a.arrivals = static_cast<unsigned long long*>(workspace);
  a.call = fa::paged_call_number();
  a.ml_part = reinterpret_cast<float2*>(static_cast<char*>(workspace) + w.ml);
  a.o_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.o);
  if (fa::device_error_word(&a.err) != FA_OK) return FA_ERR_CUDA;
  return fa::launch_paged(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_rotary_packed(const fa_rotary_call* c) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  return fa_rotary(c->x, c->x_strides, c->y, c->y_strides, c->B, c->H, c->N, c->d, c->positions, c->position_stride,
                   c->inv_freq, c->rotary_dim, c->interleaved, c->mscale, static_cast<fa_dtype>(c->dtype), c->stream);
}

fa_status fa_rotary_backward_packed(const fa_rotary_call* c) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  return fa_rotary_backward(c->x, c->x_strides, c->y, c->y_strides, c->B, c->H, c->N, c->d, c->positions,
                            c->position_stride, c->inv_freq, c->rotary_dim, c->interleaved, c->mscale,
                            static_cast<fa_dtype>(c->dtype), c->stream);
}

fa_status fa_append_paged_packed(const fa_append_paged_call* c) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  return fa_append_paged(&c->cache, c->k, c->k_strides, c->v, c->v_strides, c->q, c->q_strides, c->q_out, c->B, c->H,
                         c->Hkv, c->T, c->d, c->q_lens, c->inv_freq, c->rotary_dim, c->interleaved, c->mscale,
                         static_cast<fa_dtype>(c->dtype), c->stream);
}

fa_status fa_forward_paged_packed(const fa_forward_paged_call* c) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  const fa_score_mod mod{c->softcap, c->alibi_slopes, nullptr};
  return fa_forward_paged(c->q, &c->cache, c->o, c->lse, c->B, c->H, c->Hkv, c->T, c->d, c->scale, c->q_lens, &mod,
                          static_cast<fa_dtype>(c->dtype), c->workspace, c->workspace_bytes, c->stream);
}

}  // extern "C"
