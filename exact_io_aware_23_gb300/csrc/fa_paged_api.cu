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

// The table and the lengths of a cache.
fa_status check_table(const fa_paged_cache* c) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  if (c->n_pages < 0 || c->max_pages < 0 || c->page_size <= 0) return FA_ERR_INVALID_ARG;
  if (c->page_size % 16 != 0 || c->page_size > fa::kMaxPageSize) return FA_ERR_UNSUPPORTED;
  if ((!c->block_table && c->max_pages > 0) || !c->kv_lens) return FA_ERR_INVALID_ARG;
  if (!aligned(c->block_table, 4) || !aligned(c->kv_lens, 4) || c->table_stride < c->max_pages) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// ... and its pages, of values of `size` bytes.
fa_status check_cache(const fa_paged_cache* c, int Hkv, int size = 2) {
  const fa_status st = check_table(c);
  if (st != FA_OK) return st;
  if (!c->k_cache || !c->v_cache || !aligned(c->k_cache, 16) || !aligned(c->v_cache, 16)) return FA_ERR_INVALID_ARG;
  const int64_t unit = 16 / size;
  if (c->token_stride % unit != 0 || (c->n_pages > 1 && c->page_stride % unit != 0) || (Hkv > 1 && c->head_stride % unit != 0))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// The pages' format, their scales and bounds.  Null: 16-bit pages, nothing else.
fa_status check_store(const fa_page_store* p, bool bounds) {
  if (p == nullptr) return FA_OK;
  if (p->format != FA_PAGES_16BIT && p->format != FA_PAGES_E4M3 && p->format != FA_PAGES_INT8) return FA_ERR_UNSUPPORTED;
  const bool bits8 = p->format != FA_PAGES_16BIT;
  if (bits8 && (!p->k_scales || !p->v_scales || !aligned(p->k_scales, 4) || !aligned(p->v_scales, 4))) return FA_ERR_INVALID_ARG;
  if (bounds && (!p->k_bounds || !p->bound_scales || !aligned(p->k_bounds, 16) || !aligned(p->bound_scales, 4)))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}
int value_bytes(const fa_page_store* p) { return p == nullptr || p->format == FA_PAGES_16BIT ? 2 : 1; }

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
  return fa_append_paged_store(cache, nullptr, k, k_strides, v, v_strides, q, q_strides, q_out, B, H, Hkv, T, d, q_lens,
                               inv_freq, rotary_dim, interleaved, mscale, dtype, stream);
}

fa_status fa_append_paged_store(const fa_paged_cache* cache, const fa_page_store* store, const void* k,
                                const int64_t k_strides[3], const void* v, const int64_t v_strides[3], const void* q,
                                const int64_t q_strides[3], void* q_out, int B, int H, int Hkv, int T, int d,
                                const int32_t* q_lens, const double* inv_freq, int rotary_dim, int interleaved,
                                float mscale, fa_dtype dtype, void* stream) {
  // without queries the number of their heads does not matter; with some there have to be heads
  if (H < 0 || (q != nullptr && H == 0 && Hkv > 0)) return FA_ERR_INVALID_ARG;
  if (q == nullptr) H = Hkv;
  fa_status st = check_sizes(B, H, Hkv, T, d);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  st = check_rotation(inv_freq, rotary_dim, mscale, d);
  if (st != FA_OK) return st;
  if (B == 0 || Hkv == 0 || T == 0) return FA_OK;
  const bool bounds = store != nullptr && store->k_bounds != nullptr;
  st = check_store(store, bounds);
  if (st != FA_OK) return st;
  st = check_cache(cache, Hkv, value_bytes(store));
  if (st != FA_OK) return st;
  // the pages are written, and so are their scales
  if (value_bytes(store) == 1 && store->k_scales == store->v_scales) return FA_ERR_INVALID_ARG;
  if (value_bytes(store) == 1 && bounds && (store->bound_scales == store->k_scales || store->bound_scales == store->v_scales))
    return FA_ERR_INVALID_ARG;
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
  if (bounds || value_bytes(store) == 1) {
    fa::StoreArgs p{};
    p.store = store->format;
    p.k_scales = store->k_scales;
    p.v_scales = store->v_scales;
    p.bounds = store->k_bounds;
    p.bound_scales = store->bound_scales;
    return fa::launch_append_store(a, p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }
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
  return fa_forward_paged_store(q, cache, nullptr, nullptr, 0, o, lse, B, H, Hkv, T, d, scale, q_lens, score, dtype,
                                workspace, workspace_bytes, stream);
}

fa_status fa_forward_paged_store(const void* q, const fa_paged_cache* cache, const fa_page_store* store,
                                 const int32_t* pages, int n_select, void* o, float* lse, int B, int H, int Hkv, int T,
                                 int d, float scale, const int32_t* q_lens, const fa_score_mod* score, fa_dtype dtype,
                                 void* workspace, size_t workspace_bytes, void* stream) {
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
  st = check_store(store, false);
  if (st != FA_OK) return st;
  st = check_cache(cache, Hkv, value_bytes(store));
  if (st != FA_OK) return st;
  if (pages != nullptr && (n_select <= 0 || !aligned(pages, 4))) return FA_ERR_INVALID_ARG;
  if (!q || !o || !lse || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(q_lens, 4))
    return FA_ERR_INVALID_ARG;
  fa::PagedArgs a{};
  a.cache = cache_args(cache);
  a.pages = pages;
  a.picks = n_select;
  // (places behind all keys are a mark of keys that do not exist)
  if (pages != nullptr && fa::paged_capacity(a.cache) >= 0x7f000000) return FA_ERR_UNSUPPORTED;
  const int span = fa::paged_span(a);
  const size_t need = fa_forward_paged_workspace_size(B, H, Hkv, T, d, span);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.B = B; a.H = H; a.Hkv = Hkv; a.T = T; a.d = d;
  a.q_lens = q_lens;
  a.scale = scale;
  a.score = mods;
  if (!fa::paged_counts(B, Hkv, H / Hkv * T, span, value_bytes(store) == 1)) return FA_ERR_UNSUPPORTED;
  if (store != nullptr) {
    a.store = store->format;
    a.k_scales = store->k_scales;
    a.v_scales = store->v_scales;
  }
  a.f16 = dtype == FA_FP16;
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

size_t fa_select_pages_workspace_size(int B, int Hkv, int max_pages, int n_select) {
  if (B <= 0 || Hkv <= 0 || max_pages <= 0 || n_select <= 0 || !fa::select_scores_first(B, Hkv, max_pages, n_select)) return 0;
  size_t arrivals;
  return fa::select_workspace(B, Hkv, max_pages, &arrivals);
}

fa_status fa_select_pages(const void* q, const fa_paged_cache* cache, const fa_page_store* store, int32_t* pages, int B,
                          int H, int Hkv, int T, int d, const int32_t* q_lens, int n_select, int first, int last,
                          fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_sizes(B, H, Hkv, T, d);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (n_select < 0 || first < 0 || last < 0) return FA_ERR_INVALID_ARG;
  if (n_select > 0x7fffffff - 4096) return FA_ERR_UNSUPPORTED;          // (threads' steps over a list end behind it)
  if (B == 0 || Hkv == 0 || n_select == 0) return FA_OK;
  if (!pages || !aligned(pages, 4)) return FA_ERR_INVALID_ARG;
  if (H == 0 || T == 0)                                     // no new tokens: -1 everywhere
    return cudaMemsetAsync(pages, 0xff, (size_t)B * Hkv * n_select * sizeof(int32_t), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK : FA_ERR_CUDA;
  if (store == nullptr) return FA_ERR_INVALID_ARG;
  st = check_table(cache);
  if (st != FA_OK) return st;
  if (cache->max_pages > fa::kMaxChoice) return FA_ERR_UNSUPPORTED;
  if (!store->k_bounds || !store->bound_scales || !aligned(store->k_bounds, 16) || !aligned(store->bound_scales, 4) || !q ||
      !aligned(q, 16) || !aligned(q_lens, 4))
    return FA_ERR_INVALID_ARG;
  const size_t need = fa_select_pages_workspace_size(B, Hkv, cache->max_pages, n_select);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
  fa::SelectArgs a{};
  a.cache = cache_args(cache);
  a.q = q;
  a.bounds = store->k_bounds;
  a.bound_scales = store->bound_scales;
  a.B = B; a.H = H; a.Hkv = Hkv; a.T = T; a.d = d;
  a.q_lens = q_lens;
  a.picks = n_select;
  a.first = first;
  a.last = last;
  a.pages = pages;
  if (need > 0) {
    size_t arrivals;
    fa::select_workspace(B, Hkv, cache->max_pages, &arrivals);
    a.scores = static_cast<float*>(workspace);
    a.arrivals = reinterpret_cast<unsigned long long*>(static_cast<char*>(workspace) + arrivals);
    a.call = fa::paged_call_number();
  }
  if (fa::device_error_word(&a.err) != FA_OK) return FA_ERR_CUDA;
  return fa::launch_select(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_assign_pages(int32_t* block_table, int64_t table_stride, int B, int max_pages, int page_size,
                          const int32_t* old_lens, const int32_t* new_lens, int32_t* free_pages, int n_free,
                          const int32_t* free_state, int32_t* free_state_out, int32_t* lens, int32_t* q_lens,
                          int64_t* slots, int32_t* positions, int T, void* stream) {
  if (B < 0 || max_pages < 0 || T < 0 || n_free < 0 || page_size <= 0 || table_stride < max_pages) return FA_ERR_INVALID_ARG;
  if (page_size % 16 != 0 || page_size > fa::kMaxPageSize) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || (int64_t)B * T > 0x7fffffff - 4096) return FA_ERR_UNSUPPORTED;     // (the blocks' runs of tokens end behind T)
  if ((!block_table && B > 0 && max_pages > 0) || !free_pages || n_free == 0 || !free_state || !free_state_out)
    return FA_ERR_INVALID_ARG;
  if (B > 0 && (!old_lens || !new_lens || !lens || !q_lens || (T > 0 && (!slots || !positions)))) return FA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)block_table, (const void*)old_lens, (const void*)new_lens, (const void*)free_pages,
                        (const void*)free_state, (const void*)free_state_out, (const void*)lens, (const void*)q_lens,
                        (const void*)positions})
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return FA_ERR_INVALID_ARG;
  fa::AssignArgs a{};
  a.table = block_table;
  a.table_stride = table_stride;
  a.B = B; a.max_pages = max_pages; a.page_size = page_size; a.T = T;
  a.old_lens = old_lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.state = free_state;
  a.state_out = free_state_out;
  a.lens = lens;
  a.q_lens = q_lens;
  a.slots = slots;
  a.positions = positions;
  if (fa::device_error_word(&a.err) != FA_OK) return FA_ERR_CUDA;
  return fa::launch_assign(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_append_paged_store_packed(const fa_append_paged_store_call* call) {
  if (call == nullptr) return FA_ERR_INVALID_ARG;
  const fa_append_paged_call* c = &call->call;
  return fa_append_paged_store(&c->cache, &call->store, c->k, c->k_strides, c->v, c->v_strides, c->q, c->q_strides, c->q_out,
                               c->B, c->H, c->Hkv, c->T, c->d, c->q_lens, c->inv_freq, c->rotary_dim, c->interleaved,
                               c->mscale, static_cast<fa_dtype>(c->dtype), c->stream);
}

fa_status fa_forward_paged_store_packed(const fa_forward_paged_store_call* call) {
  if (call == nullptr) return FA_ERR_INVALID_ARG;
  const fa_forward_paged_call* c = &call->call;
  const fa_score_mod mod{c->softcap, c->alibi_slopes, nullptr};
  return fa_forward_paged_store(c->q, &c->cache, &call->store, call->pages, call->n_select, c->o, c->lse, c->B, c->H, c->Hkv, c->T, c->d,
                                c->scale, c->q_lens, &mod, static_cast<fa_dtype>(c->dtype), c->workspace,
                                c->workspace_bytes, c->stream);
}

fa_status fa_select_pages_packed(const fa_select_pages_call* c) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  return fa_select_pages(c->q, &c->cache, &c->store, c->pages, c->B, c->H, c->Hkv, c->T, c->d, c->q_lens, c->n_select,
                         c->first, c->last, static_cast<fa_dtype>(c->dtype), c->workspace, c->workspace_bytes, c->stream);
}

fa_status fa_assign_pages_packed(const fa_assign_pages_call* c) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  return fa_assign_pages(c->block_table, c->table_stride, c->B, c->max_pages, c->page_size, c->old_lens, c->new_lens,
                         c->free_pages, c->n_free, c->free_state, c->free_state_out, c->lens, c->q_lens, c->slots,
                         c->positions, c->T, c->stream);
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
