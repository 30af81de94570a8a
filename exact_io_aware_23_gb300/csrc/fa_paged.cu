// Attention of a few new tokens over a paged cache: decoding, and checking drafted tokens.
//
//     s_ij = cap(scale q_i . k_j) - slope |i - j|,  O_i = sum_j softmax_j(s_ij) v_j
//
// What bounds it: the cache's bytes.  Each key and value is read once for all G = H / Hkv query
// heads (and T new tokens) of its group; the two products are 4 * G * T flops a value, far below
// the tensor cores' share even with the rows padded to the 16 of one mma.
//
// Work.  The cache of every (sequence, key head, block of 16 query rows) is cut into tiles of 16
// keys, numbered through, and the CTAs take equal consecutive shares of the whole (their number is
// fixed by the device, the shares by the lengths, which live on the device).  A share may end
// inside a sequence: its statistics (m, l) and un-normalised output then go to the workspace, and
// a second kernel joins them in the order of the tiles.  So one long sequence fills the GPU like a
// hundred short ones, unequal lengths leave nobody idle, and every result has one fixed order of
// additions.
//
// Inside a CTA the four warps take the tiles in turn.  A warp copies its own tiles into its own
// ring in shared memory (16-byte cp.async, several tiles ahead, running on into the next sequence)
// and waits for nobody until the end of a (sequence, head); there the warps' statistics are joined
// in shared memory.  A tile lies in one page (pages are multiples of 16 tokens); rows behind the
// last key are filled with zeros, so that nothing a page holds beyond the sequence enters.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "fa_paged.cuh"
#include "fa_score.cuh"
#include "fa_sm103.cuh"
#include "ptx_sm103.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;                  // query rows of a block: one mma's
constexpr int kKeys = 16;                  // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kHalf = kKeys * kRowBytes;             // a tile's keys (or values)
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = D == 128 ? 5 : 10;           // 160 KB of tiles a CTA
  static constexpr int kRing = kStages * kStage;              // per warp
  static constexpr int kPitch = D + 8;                        // floats of a row to be joined
  static constexpr int kJoin = kWarps * kRing;
  static constexpr int kStat = kJoin + kWarps * kRows * kPitch * 4;
  static constexpr int kSmem = kStat + kWarps * kRows * 8;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;            // 0: the 16 bytes are filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// c (16 x 8, fp32) += a (16 x 16) b (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Tiles of sequence b, per key head and row block.
__device__ __forceinline__ int tiles_of(const PagedArgs& a, int b, int* err) {
  if (new_tokens(a.q_lens, b, a.T) == 0) return 0;
  return (paged_len(a.cache, b, err) + kKeys - 1) / kKeys;
}

// The tiles of all sequences, and where sequence `b` (or tile `at`) lies among them; every warp
// reckons for itself.
struct Place {
  int b;              // sequence
  int64_t before;     // tiles before it
};
__device__ __forceinline__ int64_t warp_total(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ int64_t all_tiles(const PagedArgs& a, int heads, int* err) {
  const int lane = threadIdx.x % 32;
  int64_t sum = 0;
  for (int b = lane; b < a.B; b += 32) sum += tiles_of(a, b, err);
  return warp_total(sum) * heads;
}
// The sequence that holds tile `at`, which is below the total.
__device__ Place find_tile(const PagedArgs& a, int heads, int64_t at) {
  const int lane = threadIdx.x % 32;
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int64_t n = b0 + lane < a.B ? (int64_t)tiles_of(a, b0 + lane, nullptr) * heads : 0;
    int64_t sum = n;                                   // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + sum > at);
    if (past != 0u) {
      const int l = __ffs(past) - 1;
      Place p;
      p.b = b0 + l;
      p.before = before + __shfl_sync(0xffffffffu, sum - n, l);
      return p;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return Place{a.B, before};
}

// CTAs that share `total` tiles: each gets at least kMinTiles (one per warp and then some: a share
// too small costs more in joining than it saves), none more than the grid has.
constexpr int kMinTiles = 8;
__host__ __device__ inline int sharing_ctas(int64_t total, int ctas) {
  const int64_t want = (total + kMinTiles - 1) / kMinTiles;
  return want < 1 ? 1 : want > ctas ? ctas : (int)want;
}
__host__ __device__ inline int64_t share_begin(int64_t total, int n, int c) { return total * c / n; }

// A (sequence, key head, row block) and a tile in it; advances over empty sequences.
struct Walk {
  int b, hr, tile, tiles, len;
  __device__ void enter(const PagedArgs& a) {          // at hr = 0 of b, or past the end
    while (b < a.B) {
      len = paged_len(a.cache, b, nullptr);
      tiles = new_tokens(a.q_lens, b, a.T) == 0 ? 0 : (len + kKeys - 1) / kKeys;
      if (tiles > 0) return;
      ++b;
    }
    tiles = 1 << 30;
  }
  __device__ void next_segment(const PagedArgs& a, int heads) {
    if (++hr == heads) {
      hr = 0;
      ++b;
      enter(a);
    }
  }
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) paged_kernel(const PagedArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = a.H / a.Hkv, rows = G * a.T;
  const int blocks = (rows + kRows - 1) / kRows;       // row blocks of a key head
  const int heads = a.Hkv * blocks;
  asm volatile("griddepcontrol.launch_dependents;");   // the joining kernel may be set up meanwhile

  const int64_t total = all_tiles(a, heads, blockIdx.x == 0 && warp == 0 ? a.err : nullptr);
  const int n_ctas = sharing_ctas(total, gridDim.x);
  if ((int)blockIdx.x >= n_ctas || total == 0) return;
  const int64_t begin = share_begin(total, n_ctas, blockIdx.x);
  const int64_t end = share_begin(total, n_ctas, blockIdx.x + 1);
  Walk seg;
  {
    const Place p = find_tile(a, heads, begin);
    seg.b = p.b;
    seg.hr = 0;
    seg.enter(a);
    const int64_t off = begin - p.before;
    seg.hr = (int)(off / seg.tiles);
    seg.tile = (int)(off % seg.tiles);
  }

  // ---- the warp's copies: tiles begin + warp, begin + warp + 4, ... into its own ring -----------
  const uint32_t ring = ptx::smem_u32(smem) + warp * C::kRing;
  Walk load = seg;
  int64_t at = begin;
  auto step = [&](int n) {                              // n tiles on
    at += n;
    if (at >= end) return;
    int t = load.tile + n;
    while (t >= load.tiles) {
      t -= load.tiles;
      load.next_segment(a, heads);
    }
    load.tile = t;
  };
  auto page_of = [&]() {
    if (at >= end) return 0;
    return a.cache.table[load.b * a.cache.table_stride + load.tile * kKeys / a.cache.page_size];
  };
  step(warp);
  int page = page_of();                                 // of the next tile to copy
  int slot = 0;
  auto copy_tile = [&]() {
    if (at < end) {
      const bool good = (unsigned)page < (unsigned)a.cache.n_pages;
      if (!good && lane == 0) atomicExch(a.err, kDevBadOffsets);      // reported, not followed
      const int first = load.tile * kKeys % a.cache.page_size;
      const int64_t base = (good ? (int64_t)page * a.cache.page_stride : 0) +
                           (int64_t)(load.hr / blocks) * a.cache.head_stride;
      const uint32_t dst = ring + slot * C::kStage;
      constexpr int kChunks = D / 8, kStep = 32 / kChunks;     // 16-byte pieces of a row; rows a step
      const int c = lane % kChunks;
      const int n = good ? load.len - load.tile * kKeys : 0;   // keys of the tile that exist
#pragma unroll
      for (int i = 0; i < kKeys / kStep; ++i) {
        const int r = i * kStep + lane / kChunks;
        const bool there = r < n;
        const int64_t off = base + (there ? (int64_t)(first + r) * a.cache.token_stride : 0) + c * 8;
        const uint32_t to = dst + r * C::kRowBytes + ((c ^ (r & 7)) << 4);
        cp16(to, static_cast<const uint16_t*>(a.cache.k) + off, there);
        cp16(to + C::kHalf, static_cast<const uint16_t*>(a.cache.v) + off, there);
      }
      step(kWarps);
      page = page_of();
    }
    cp_commit();
    slot = slot + 1 == C::kStages ? 0 : slot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages - 1; ++i) copy_tile();

  // ---- the warp's products -----------------------------------------------------------------------
  const int r0 = lane / 4, c0 = (lane % 4) * 2;
  const float c_log2 = a.scale * kLog2e;
  float* const join = reinterpret_cast<float*>(smem + C::kJoin);
  float2* const stat = reinterpret_cast<float2*>(smem + C::kStat);
  int take = 0;                                         // ring slot of the next tile
  int turn = 0;                                         // the warp whose turn the segment's first tile is
#pragma unroll 1
  for (int64_t g = begin; g < end;) {
    const int n = (int)min((int64_t)(seg.tiles - seg.tile), end - g);
    const int block = seg.hr % blocks, hk = seg.hr / blocks;
    const int row0 = block * kRows;                     // first row of the block in the group
    const int n_rows = min(kRows, rows - row0);
    const int count = new_tokens(a.q_lens, seg.b, a.T);
    const int64_t qrow = ((int64_t)seg.b * a.H + hk * G) * a.T + row0;
    const int mine = (warp - turn + kWarps) % kWarps;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    if (mine < n) {
      // the block's queries as mma operands, and each row's place, slope
      uint32_t q[D / 16][4];
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + qrow * D);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + (e & 1) * 8;
          q[i][e] = r < n_rows ? __ldg(qp + (r * D + i * 16 + (e >> 1) * 8 + c0) / 2) : 0u;
        }
      int limit[2];                                     // keys that the row sees
      float slope[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row0 + r0 + e * 8, t = r % a.T;
        limit[e] = r < rows && t < count ? seg.len - count + t + 1 : 0;
        slope[e] = a.score.slopes != nullptr && r < rows ? a.score.slopes[hk * G + r / a.T] * kLog2e : 0.f;
      }
#pragma unroll 1
      for (int i = mine; i < n; i += kWarps) {
        cp_wait<C::kStages - 2>();
        __syncwarp();                                   // this tile is there, the last one read
        copy_tile();                                    // into the last one's slot
        const uint32_t ks = ring + take * C::kStage, vs = ks + C::kHalf;
        take = take + 1 == C::kStages ? 0 : take + 1;
        float s[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[h][e] = 0.f;
        {
          // matrices of the load: keys 0-7 and 8-15, two groups of 8 values each
          const int key = (lane & 7) + ((lane >> 4) << 3), part = (lane >> 3) & 1;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldsm4(ks + key * C::kRowBytes + (((2 * k + part) ^ (key & 7)) << 4), b);
            mma<F16>(s[0], q[k], b[0], b[1]);
            mma<F16>(s[1], q[k], b[2], b[3]);
          }
        }
        // scores in the log2 domain, masked
        const int key0 = (seg.tile + i) * kKeys;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + h * 8 + c0 + (e & 1);
            const int lim = limit[e >> 1];
            float x = s[h][e];
            x = a.score.cap_log2 != 0.f ? a.score.cap_log2 * tanh_one(x, a.score) : x * c_log2;
            x = fmaf(slope[e >> 1], (float)(key - (lim - 1)), x);
            s[h][e] = key < lim ? x : -INFINITY;
          }
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[e], mx);
          const float sub = mn == -INFINITY ? 0.f : mn;
          const float alpha = ptx::ex2(m[e] - sub);       // 0 while the row is empty
          m[e] = mn;
          float p0 = ptx::ex2(s[0][2 * e] - sub), p1 = ptx::ex2(s[0][2 * e + 1] - sub);
          float p2 = ptx::ex2(s[1][2 * e] - sub), p3 = ptx::ex2(s[1][2 * e + 1] - sub);
          l[e] = l[e] * alpha + ((p0 + p1) + (p2 + p3));
          p[e] = ptx::pack2<F16>(p0, p1);
          p[e + 2] = ptx::pack2<F16>(p2, p3);
          if (alpha != 1.f) {
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
              o[k][2 * e] *= alpha;
              o[k][2 * e + 1] *= alpha;
            }
          }
        }
        {
          const int key = lane & 15, part = lane >> 4;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldsm4t(vs + key * C::kRowBytes + (((2 * k + part) ^ (key & 7)) << 4), b);
            mma<F16>(o[2 * k], p, b[0], b[1]);
            mma<F16>(o[2 * k + 1], p, b[2], b[3]);
          }
        }
      }
    }
    // ---- the segment's end: join the warps -------------------------------------------------------
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    if (lane % 4 == 0) {
      stat[warp * kRows + r0] = make_float2(m[0], l[0]);
      stat[warp * kRows + r0 + 8] = make_float2(m[1], l[1]);
    }
    if (mine < n) {
      float* to = join + (warp * kRows + r0) * C::kPitch + c0;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        *reinterpret_cast<float2*>(to + k * 8) = make_float2(o[k][0], o[k][1]);
        *reinterpret_cast<float2*>(to + 8 * C::kPitch + k * 8) = make_float2(o[k][2], o[k][3]);
      }
    }
    __syncthreads();
    {
      const bool whole = n == seg.tiles;
      const int64_t part = 2 * (int64_t)blockIdx.x + (g == begin ? 0 : 1);
      constexpr int kQuads = D / 4;
      for (int x = threadIdx.x; x < n_rows * kQuads; x += kThreads) {
        const int r = x / kQuads, c = x % kQuads * 4;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, stat[w * kRows + r].x);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mx != -INFINITY) {
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 ml = stat[w * kRows + r];
            if (ml.x == -INFINITY) continue;
            const float f = ptx::ex2(ml.x - mx);
            const float4 v = *reinterpret_cast<const float4*>(join + (w * kRows + r) * C::kPitch + c);
            sum = fmaf(f, ml.y, sum);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
          }
        }
        if (whole) {
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          const uint2 w = make_uint2(ptx::pack2<F16>(acc.x * inv, acc.y * inv), ptx::pack2<F16>(acc.z * inv, acc.w * inv));
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + (qrow + r) * D + c) = w;
          if (c == 0) a.lse[qrow + r] = sum > 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
        } else {
          *reinterpret_cast<float4*>(a.o_part + (part * kRows + r) * D + c) = acc;
          if (c == 0) a.ml_part[part * kRows + r] = make_float2(mx, sum);
        }
      }
    }
    __syncthreads();
    turn = (turn + n) % kWarps;
    g += n;
    seg.tile = 0;
    if (g < end) seg.next_segment(a, heads);
  }
  cp_wait<0>();
}

// Joins the parts of every segment that several CTAs shared, in the order of the tiles, and writes
// the rows of sequences without keys.  One CTA per (sequence, key head, row block).
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const PagedArgs a) {
  const int G = a.H / a.Hkv, rows = G * a.T;
  const int blocks = (rows + kRows - 1) / kRows, heads = a.Hkv * blocks;
  const int b = blockIdx.x / heads, hr = blockIdx.x % heads;
  const int block = hr % blocks, hk = hr / blocks;
  const int row0 = block * kRows, n_rows = min(kRows, rows - row0);
  const int64_t qrow = ((int64_t)b * a.H + hk * G) * a.T + row0;
  const int tiles = tiles_of(a, b, nullptr);
  constexpr int kQuads = D / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tiles == 0) {
    for (int x = threadIdx.x; x < n_rows * kQuads; x += kThreads) {
      const int r = x / kQuads, c = x % kQuads * 4;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + (qrow + r) * D + c) = make_uint2(0u, 0u);
      if (c == 0) a.lse[qrow + r] = -INFINITY;
    }
    return;
  }
  const int lane = threadIdx.x % 32;
  int64_t sum = 0, first = 0;                          // all tiles; those before this sequence
  for (int i = lane; i < a.B; i += 32) {
    const int64_t n = tiles_of(a, i, nullptr);
    sum += n;
    if (i < b) first += n;
  }
  const int64_t total = warp_total(sum) * heads;
  const int64_t s0 = warp_total(first) * heads + (int64_t)hr * tiles, s1 = s0 + tiles;
  const int n_ctas = sharing_ctas(total, a.ctas);
  auto owner = [&](int64_t t) {                        // the CTA whose share holds tile t
    int c = (int)(t * n_ctas / total);
    while (share_begin(total, n_ctas, c + 1) <= t) ++c;
    while (share_begin(total, n_ctas, c) > t) --c;
    return c;
  };
  const int ca = owner(s0), cb = owner(s1 - 1);
  if (ca == cb) return;                                // one CTA had it all and wrote it
  // the first CTA may have begun inside an earlier segment: this one is then its last
  const int64_t part0 = 2 * (int64_t)ca + (share_begin(total, n_ctas, ca) == s0 ? 0 : 1);
  for (int x = threadIdx.x; x < n_rows * kQuads; x += kThreads) {
    const int r = x / kQuads, c = x % kQuads * 4;
    float mx = -INFINITY;
    for (int i = ca; i <= cb; ++i)
      mx = fmaxf(mx, __ldcg(&a.ml_part[(i == ca ? part0 : 2 * (int64_t)i) * kRows + r]).x);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mx != -INFINITY) {
#pragma unroll 4
      for (int i = ca; i <= cb; ++i) {
        const int64_t p = (i == ca ? part0 : 2 * (int64_t)i) * kRows + r;
        const float2 ml = __ldcg(&a.ml_part[p]);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.o_part + p * D + c));
        const float f = ptx::ex2(ml.x - mx);           // 0 for a part without keys
        l = fmaf(f, ml.y, l);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const uint2 w = make_uint2(ptx::pack2<F16>(acc.x * inv, acc.y * inv), ptx::pack2<F16>(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + (qrow + r) * D + c) = w;
    if (c == 0) a.lse[qrow + r] = l > 0.f ? (mx + log2f(l)) * kLn2 : -INFINITY;
  }
}

template <int D, bool F16>
cudaError_t paged(const PagedArgs& a, cudaStream_t s) {
  auto kern = paged_kernel<D, F16>;
  static LaunchSetup setup;
  cudaError_t e = prepare_launch(setup, kern, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<a.ctas, kThreads, Cfg<D>::kSmem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int rows = a.H / a.Hkv * a.T;
  const int64_t segments = (int64_t)a.B * a.Hkv * ((rows + kRows - 1) / kRows);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)segments);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, F16>, a);
}

}  // namespace

int paged_ctas(int d) {
  int sms = 0;
  (void)d;
  return sm_count(&sms) == cudaSuccess && sms > 0 ? sms : 152;   // GB300's when no device can be asked
}

size_t paged_parts(int ctas) { return 2 * (size_t)ctas * kRows; }

size_t paged_workspace(int d) {
  const size_t parts = paged_parts(paged_ctas(d));
  return parts * d * sizeof(float) + parts * sizeof(float2);
}

cudaError_t launch_paged(const PagedArgs& a, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_FP16) return a.d == 64 ? paged<64, true>(a, s) : paged<128, true>(a, s);
  return a.d == 64 ? paged<64, false>(a, s) : paged<128, false>(a, s);
}

}  // namespace fa
