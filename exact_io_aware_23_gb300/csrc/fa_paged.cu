// Attention of a few new tokens over a paged cache: decoding, and checking drafted tokens.
//
//     s_ij = cap(scale q_i . k_j) - slope |i - j|,  O_i = sum_j softmax_j(s_ij) v_j
//
// What bounds it: the cache's bytes.  Each key and value is read once for all G = H / Hkv query
// heads (and T new tokens) of its group; the two products are 4 * G * T flops a value, far below
// the tensor cores' share even with the rows padded to the 16 of one mma.  (So the warps feed
// mma.sync from shared memory themselves; a 128-row tile of the fifth-generation cores would be
// nearly all padding.)  Measured: B2 H32 Hkv8 d128 with 119K and 131K keys, 1.03 GB: 160 us, 6.4 TB/s,
// 0.96 of the copy rate; 64 sequences of 1 to 8192 keys, 1.02 GB: 161 us; 16 sequences of up to 4000
// keys at d = 64, five drafted tokens: 37 us, 4.1 TB/s (there the warps' own work shows).
//
// Work.  The cache of every (sequence, key head, block of 16 query rows), a segment, is cut into tiles
// of 16 or 32 keys, numbered through, and the CTAs take equal consecutive shares of the whole (their
// number is fixed by the device, the shares by the lengths, which live on the device).  A share may
// end inside a segment: its statistics (m, l) and un-normalised output then go to the workspace, and
// the CTA that finishes a segment last joins its parts, in the order of the tiles.  So one long
// sequence fills the GPU like a hundred short ones, unequal lengths leave nobody idle, and every
// result has one fixed order of additions.
//
// Inside a CTA the four warps take the tiles in turn.  A warp copies its own tiles into its own
// ring in shared memory (16-byte cp.async, several tiles ahead, running on into the next segment)
// and waits for nobody until the end of a segment; there the warps' statistics are joined in shared
// memory.  16 keys lie in one page (pages are multiples of 16 tokens); rows behind the last key are
// filled with zeros, so that nothing a page holds beyond the sequence enters.  P is rounded to the
// values' type for its product, like theirs an error of half a step; l, m, O stay in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>
#include <chrono>

#include "fa_paged.cuh"
#include "fa_score.cuh"
#include "fa_sm103.cuh"
#include "ptx_sm103.cuh"

namespace fa {
namespace {

// Four warps a CTA and two CTAs an SM: eight warps hide each other's latencies, and two segments' ends
// (queries, join) overlap.  (B64 H32 Hkv8 d128, 1 to 8192 keys: 163 us, against 181 with eight warps in
// one CTA; B256 with 1 to 200 keys: 65 against 98.  Four CTAs of two warps: about the same there, but
// twice the parts to join of a long cache, 182 us against 164 for B2 of 128K keys.)
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Query rows of a block: one mma's.  A group of more rows (T new tokens of H / Hkv heads) takes several
// blocks, each reading the cache (through L2) again; blocks of two mma's rows read it half as often but
// hold twice the output in registers and spill (B8 H64 Hkv8 T7 d128, 4096 keys: 95 us against 74).
constexpr int kRows = 16;
constexpr int kCtasPerSm = 8 / kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;       // the running maximum is raised when a score exceeds it by more

template <int D>
struct Cfg {
  static constexpr int kKeys = D == 128 ? 16 : 32;            // keys of a tile: 8 KB with the values
  static constexpr int kParts = kKeys / 16;                   // 16-key parts of a tile, each in one page
  static constexpr int kRowBytes = D * 2;
  static constexpr int kHalf = kKeys * kRowBytes;             // a tile's keys (or values)
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = 192 * 1024 / kCtasPerSm / (kWarps * kStage);   // 192 KB of tiles an SM
  static constexpr int kRing = kStages * kStage;              // per warp
  static constexpr int kStat = kWarps * kRing;
  static constexpr int kFrom = kStat + kWarps * kRows * 8;
  static constexpr int kParted = kFrom + kWarps * 4 + 16;       // after a flag: statistics to be joined
  static constexpr int kJoin = 64;                              // parts
  static constexpr int kSmem = kParted + kJoin * kRows * 8;
  static_assert(kStage >= kRows * D * 4, "a warp's output to be joined fits the slot of its last tile");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;            // 0: the 16 bytes are filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ void mma(float* c, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---- sharing the work ------------------------------------------------------------------------------
//
// A segment is one (sequence, key head, row block).  It counts kSegment units for what it costs
// whatever its length (its queries, the join of the warps; about as long as the CTA takes for that
// many tiles), then one per tile; unit numbers run over all segments, and each CTA takes an equal
// range of them.
constexpr int kSegment = 4;
constexpr int kMinUnits = kSegment + kWarps;   // a smaller share costs more in joining than it saves

__host__ __device__ inline int sharing_ctas(int units, int ctas) {
  const int want = (units + kMinUnits - 1) / kMinUnits;
  return want < 1 ? 1 : want > ctas ? ctas : want;
}
// CTA c's range begins at c * q + min(c, r) for units = n * q + r
struct Shares {
  int q, r;
  __device__ Shares(int units, int n) : q(units / n), r(units % n) {}
  __device__ int begin(int c) const { return c * q + min(c, r); }
  __device__ int owner(int u) const { return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q; }
};

template <int kKeys>
__device__ __forceinline__ int tiles_of(const PagedArgs& a, int b, int* err) {
  if (new_tokens(a.q_lens, b, a.T) == 0) return 0;
  return (paged_len(a.cache, b, err) + kKeys - 1) / kKeys;
}
template <int kKeys>
__device__ __forceinline__ int units_of(const PagedArgs& a, int heads, int b, int* err) {
  const int n = b < a.B ? tiles_of<kKeys>(a, b, err) : 0;
  return n > 0 ? (n + kSegment) * heads : 0;
}

// A warp's reckoning of all sequences' units: the first 256 sequences' stay in registers (all their
// lengths are read at once), further ones are read again.
template <int kKeys>
struct Reckoning {
  int keep[8];
  int total;
  __device__ Reckoning(const PagedArgs& a, int heads, int* err) {
    const int lane = threadIdx.x % 32;
    int sum = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      keep[c] = units_of<kKeys>(a, heads, c * 32 + lane, err);
      sum += keep[c];
    }
    for (int b = 256 + lane; b < a.B; b += 32) sum += units_of<kKeys>(a, heads, b, err);
    total = __reduce_add_sync(0xffffffffu, sum);
  }
  // The sequence that holds unit u, and the units before it.
  __device__ void find(const PagedArgs& a, int heads, int u, int* b, int* before) const {
    const int lane = threadIdx.x % 32;
    int done = 0;
    auto chunk = [&](int n, int b0) {
      int sum = n;                                     // inclusive scan
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, done + sum > u);
      if (past != 0u) {
        const int l = __ffs(past) - 1;
        *b = b0 + l;
        *before = done + __shfl_sync(0xffffffffu, sum - n, l);
        return true;
      }
      done += __shfl_sync(0xffffffffu, sum, 31);
      return false;
    };
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (chunk(keep[c], c * 32)) return;
    for (int b0 = 256; b0 < a.B; b0 += 32)
      if (chunk(units_of<kKeys>(a, heads, b0 + lane, nullptr), b0)) return;
  }
};

// A segment and a tile in it.  The next sequence's lengths are read ahead.
template <int kKeys>
struct Walk {
  int b, hk, block, tile, tiles, len, count;
  int ahead_len, ahead_q;                              // of sequence b + 1, as stored
  __device__ void read_ahead(const PagedArgs& a) {
    const int n = b + 1;
    ahead_len = n < a.B ? a.cache.kv_lens[n] : 0;
    ahead_q = n < a.B && a.q_lens != nullptr ? a.q_lens[n] : a.T;
  }
  __device__ void take(const PagedArgs& a, int kv, int q) {
    len = kv > paged_capacity(a.cache) ? 0 : max(kv, 0);
    count = min(max(q, 0), a.T);
    tiles = count == 0 ? 0 : (len + kKeys - 1) / kKeys;
  }
  __device__ void start(const PagedArgs& a, int seq) {
    b = seq;
    hk = block = tile = 0;
    take(a, a.cache.kv_lens[b], a.q_lens != nullptr ? a.q_lens[b] : a.T);
    read_ahead(a);
  }
  // to the next segment with tiles; past the last one, tiles is beyond any tile number
  __device__ void next(const PagedArgs& a, int blocks) {
    if (++block < blocks) return;
    block = 0;
    if (++hk < a.Hkv) return;
    hk = 0;
    do {
      ++b;
      if (b >= a.B) {
        tiles = 1 << 30;
        return;
      }
      take(a, ahead_len, ahead_q);
      read_ahead(a);
    } while (tiles == 0);
  }
};

// O = 0 and LSE = -inf for rows [row, row + n)
template <int D>
__device__ __forceinline__ void no_keys(const PagedArgs& a, int64_t row, int n) {
  for (int x = threadIdx.x; x < n * (D / 4); x += kThreads) {
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * D)[x] = make_uint2(0u, 0u);
    if (x < n) a.lse[row + x] = -INFINITY;
  }
}

template <int D, bool F16>
__device__ __forceinline__ void write_row4(const PagedArgs& a, int64_t row, int c, float4 acc, float sum, float mx) {
  const float inv = sum != 0.f ? 1.f / sum : 0.f;        // 0: no key; NaN stays
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * D + c) =
      make_uint2(ptx::pack2<F16>(acc.x * inv, acc.y * inv), ptx::pack2<F16>(acc.z * inv, acc.w * inv));
  if (c == 0) a.lse[row] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// Announces this CTA's part of a segment that CTAs ca..cb share, and says whether all of them are
// there; run by one warp.  Every part has a word of its own, set to the call's number: no atomic
// that 38 CTAs contend for (counting them in one word by compare-and-swap took 18 us at the end of
// B1 H32 Hkv8 with 32K keys).  Between its own store and its reads of the others each CTA has a
// sequentially consistent fence, so the last of them sees all words set, or cleared by one that did;
// should two see them, both join the parts, to the same bits.  Who joins clears the words, for a
// captured call's next run under the same number (another that reads them cleared has nothing left
// to do).  Whatever else a fresh workspace holds is not the number: it has 64 bits, starts at another
// place in every process, and is not used twice in one.  So no launch is spent on clearing the words
// first.  (By cudaMemsetAsync: 3 us of a call's 40.)
__device__ __forceinline__ bool all_arrived(unsigned long long* words, int mine, int part0, int ca, int cb,
                                            unsigned long long call) {
  const int lane = threadIdx.x % 32;
  if (lane == 0) {
    // releases what the whole CTA wrote before its barrier
    asm volatile("fence.acq_rel.gpu;" ::: "memory");
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(words + mine), "l"(call) : "memory");
  }
  __syncwarp();
  asm volatile("fence.sc.gpu;" ::: "memory");
  bool there = true;
  for (int i = ca + lane; i <= cb; i += 32) {
    unsigned long long w;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(words + (i == ca ? part0 : 2 * i)) : "memory");
    there = there && w == call;
  }
  there = __all_sync(0xffffffffu, there);
  if (there) asm volatile("fence.acq_rel.gpu;" ::: "memory");     // the parts, for the CTA after its barrier
  return there;
}

// kShared: CTAs share all segments' units.  Otherwise a CTA has one segment to itself (few short
// ones: nothing to join, nothing to reckon).
template <int D, bool F16, bool kShared>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_kernel(const PagedArgs a) {
  using C = Cfg<D>;
  constexpr int kKeys = C::kKeys, kParts = C::kParts, kQuads = D / 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = a.H / a.Hkv, rows = G * a.T;
  const int blocks = (rows + kRows - 1) / kRows;       // row blocks of a key head
  const int heads = a.Hkv * blocks;

  Walk<kKeys> seg;
  int units = 0, n_ctas = 1, s0 = 0;                   // s0: the segment's first unit
  int begin = 0, end = 0;                              // the CTA's units
  if constexpr (kShared) {
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
      if (tiles_of<kKeys>(a, b, nullptr) == 0) no_keys<D>(a, (int64_t)b * a.H * a.T, a.H * a.T);
    const Reckoning<kKeys> all(a, heads, blockIdx.x == 0 && warp == 0 ? a.err : nullptr);
    units = all.total;
    n_ctas = sharing_ctas(units, gridDim.x);
    if ((int)blockIdx.x >= n_ctas || units == 0) return;
    const Shares share(units, n_ctas);
    begin = share.begin(blockIdx.x);
    end = share.begin(blockIdx.x + 1);
    int b, before;
    all.find(a, heads, begin, &b, &before);
    seg.start(a, b);
    const int hr = (begin - before) / (seg.tiles + kSegment);
    seg.hk = hr / blocks;
    seg.block = hr % blocks;
    s0 = before + hr * (seg.tiles + kSegment);
    seg.tile = max(0, begin - s0 - kSegment);
  } else {
    const int hr = blockIdx.x % heads;
    seg.start(a, blockIdx.x / heads);
    seg.hk = hr / blocks;
    seg.block = hr % blocks;
    if (blockIdx.x % heads == 0 && threadIdx.x == 0) paged_len(a.cache, seg.b, a.err);
    if (seg.tiles == 0) {
      no_keys<D>(a, ((int64_t)seg.b * a.H + seg.hk * G) * a.T + seg.block * kRows, min(kRows, rows - seg.block * kRows));
      return;
    }
    end = seg.tiles + kSegment;
  }
  // tiles of the current segment up to this number are the CTA's
  auto last_tile = [&](int first_unit, int tiles) { return min(tiles, end - first_unit - kSegment); };

  // ---- the warp's copies: every fourth tile of the CTA's, into its own ring ----------------------
  const uint32_t ring = ptx::smem_u32(smem) + warp * C::kRing;
  Walk<kKeys> load = seg;
  int load_s0 = s0;
  bool more = true;
  auto step = [&](int n) {                              // n tiles on
    int t = load.tile + n;
    while (t >= load.tiles) {
      t -= load.tiles;
      load_s0 += load.tiles + kSegment;
      load.next(a, blocks);
      if (load_s0 + kSegment >= end) break;
    }
    load.tile = t;
    more = load_s0 + kSegment + t < end;
  };
  // The next tile's parts of 16 keys: their pages, and their first rows in them.  parts / (parts of
  // a page) by multiplication with the rounded-up reciprocal, exact for the sizes the host admits.
  int page[kParts], first[kParts];
  auto read_pages = [&]() {
    if (!more) return;
    const int32_t* row = a.cache.table + load.b * a.cache.table_stride;
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
      const uint32_t part = load.tile * kParts + x;
      const uint32_t at = (uint32_t)(((uint64_t)part * a.parts_magic) >> 36);
      first[x] = (int)(part - at * a.page_parts) * 16;
      page[x] = x == 0 || (int)part * 16 < load.len ? row[at] : 0;
    }
  };
  more = s0 + kSegment + seg.tile < end;
  if (more) step(warp);
  read_pages();
  // This lane's 16-byte pieces: column c of rows row, row + kStep, ...; in shared memory piece c of
  // row r lies at r * kRowBytes + ((c ^ (r & 7)) << 4), so that eight rows' pieces fill all banks.
  constexpr int kChunks = D / 8, kStep = 32 / kChunks;
  const int lane_row = lane / kChunks, lane_col = lane % kChunks;
  const uint32_t lane_off = lane_row * C::kRowBytes + ((lane_col ^ lane_row) << 4);
  const uint16_t* const kbase = static_cast<const uint16_t*>(a.cache.k) + lane_col * 8;
  const int64_t v_off = static_cast<const uint16_t*>(a.cache.v) - static_cast<const uint16_t*>(a.cache.k);
  const int64_t row_step = kStep * a.cache.token_stride;
  int slot = 0;
  auto copy_tile = [&]() {
    if (more) {
      const uint32_t dst = ring + slot * C::kStage + lane_off;
#pragma unroll
      for (int x = 0; x < kParts; ++x) {
        int n = load.len - (load.tile * kParts + x) * 16;      // keys of the part that exist
        if ((unsigned)page[x] >= (unsigned)a.cache.n_pages && n > 0) {
          if (lane == 0) atomicExch(a.err, kDevBadOffsets);    // reported, not followed
          n = 0;
        }
        const uint16_t* src = kbase;
        if (n > 0)
          src += page[x] * a.cache.page_stride + load.hk * a.cache.head_stride + (first[x] + lane_row) * a.cache.token_stride;
        if (n >= 16) {
#pragma unroll
          for (int i = 0; i < 16 / kStep; ++i, src += row_step) {
            const uint32_t to = (dst ^ (((i * kStep) & 7) << 4)) + (x * 16 + i * kStep) * C::kRowBytes;
            cp16(to, src);
            cp16(to + C::kHalf, src + v_off);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16 / kStep; ++i, src += row_step) {
            const bool there = i * kStep + lane_row < n;
            const uint16_t* from = there ? src : kbase;
            const uint32_t to = (dst ^ (((i * kStep) & 7) << 4)) + (x * 16 + i * kStep) * C::kRowBytes;
            cp16(to, from, there);
            cp16(to + C::kHalf, from + v_off, there);
          }
        }
      }
      step(kWarps);
      read_pages();
    }
    cp_commit();
    slot = slot + 1 == C::kStages ? 0 : slot + 1;
  };

  // ---- the warp's products -----------------------------------------------------------------------
  const int r0 = lane / 4, c0 = (lane % 4) * 2;
  const float c_log2 = a.scale * kLog2e;
  float2* const stat = reinterpret_cast<float2*>(smem + C::kStat);
  int* const from = reinterpret_cast<int*>(smem + C::kFrom);   // where each warp's output to be joined lies
  int* const flag = from + kWarps;
  float2* const joined = reinterpret_cast<float2*>(smem + C::kParted);
  int take = 0;                                         // ring slot of the next tile
  int turn = 0;                                         // the warp whose turn the segment's first tile is
  bool first_seg = true;

  // the segment's queries as mma operands; per row its slope and the keys it sees
  uint32_t q[D / 16][4];
  int limit[2], full;
  float slope[2];
  auto read_rows = [&]() {
    const int row0 = seg.block * kRows, n_rows = min(kRows, rows - row0);
    const int64_t qrow = ((int64_t)seg.b * a.H + seg.hk * G) * a.T + row0;
    const uint32_t* qp = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + qrow * D + r0 * D + c0);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        q[i][e] = r0 + (e & 1) * 8 < n_rows ? __ldg(qp + ((e & 1) * 8 * D + i * 16 + (e >> 1) * 8) / 2) : 0u;
    full = 0x7fffffff;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + r0 + e * 8;
      const int h = a.T == 1 ? r : r / a.T, t = r - h * a.T;
      limit[e] = r < rows && t < seg.count ? seg.len - seg.count + t + 1 : 0;
      if (r < rows) full = min(full, limit[e]);
      slope[e] = a.score.slopes != nullptr && r < rows ? __ldg(a.score.slopes + seg.hk * G + h) * kLog2e : 0.f;
    }
    full = __reduce_min_sync(0xffffffffu, full);        // keys that every row sees
  };
  read_rows();                                          // before the copies fill the way to memory
#pragma unroll 1
  for (int i = 0; i < C::kStages - 1; ++i) copy_tile();

#pragma unroll 1
  while (s0 + kSegment < end) {
    const int n = last_tile(s0, seg.tiles) - seg.tile;  // the CTA's tiles of the segment: at least one
    const int mine = (warp - turn + kWarps) % kWarps;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll 1
    for (int i = mine; i < n; i += kWarps) {
      cp_wait<C::kStages - 2>();
      __syncwarp();                                   // this tile is there, the last one read
      copy_tile();                                    // into the last one's slot
      const uint32_t ks = ring + take * C::kStage, vs = ks + C::kHalf;
      take = take + 1 == C::kStages ? 0 : take + 1;
      constexpr int kN = kKeys / 8;                     // groups of 8 keys
      float s[kKeys / 2];                               // row r0: s[4 n], s[4 n + 1]; r0 + 8: the next two
#pragma unroll
      for (int e = 0; e < kKeys / 2; ++e) s[e] = 0.f;
      {
        // matrices of a load: keys 0-7 and 8-15, two groups of 8 values each
        const int key = (lane & 7) + ((lane >> 4) << 3), part = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < kParts; ++x) {
            uint32_t b[4];
            ldsm4(ks + (x * 16 + key) * C::kRowBytes + (((2 * k + part) ^ (key & 7)) << 4), b);
            mma<F16>(&s[8 * x], q[k], b[0], b[1]);
            mma<F16>(&s[8 * x + 4], q[k], b[2], b[3]);
          }
      }
      // scores in the log2 domain
      const int key0 = (seg.tile + i) * kKeys;
      if (a.score.cap_log2 == 0.f) {
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e) s[e] *= c_log2;
      } else if (poly_fits(s, a.score.poly_limit)) {
#pragma unroll
        for (int e = 0; e < kKeys / 2; e += 2) {
          const float2 t = tanh_poly(make_float2(s[e], s[e + 1]), a.score);
          s[e] = t.x * a.score.cap_log2;
          s[e + 1] = t.y * a.score.cap_log2;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e) s[e] = a.score.cap_log2 * tanh_one(s[e], a.score);
      }
      if (a.score.slopes != nullptr) {
        float ahead[2];                                 // minus the distance at the lane's first key, exact
#pragma unroll
        for (int e = 0; e < 2; ++e) ahead[e] = (float)(key0 + c0 - (limit[e] - 1));
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e)
          s[e] = fmaf(slope[(e >> 1) & 1], ahead[(e >> 1) & 1] + (float)((e >> 2) * 8 + (e & 1)), s[e]);
      }
      if (key0 + kKeys > full) {                        // some row does not see all of the tile
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e)
          s[e] = key0 + (e >> 2) * 8 + c0 + (e & 1) < limit[(e >> 1) & 1] ? s[e] : -INFINITY;
      }
      uint32_t p[kParts][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(s[2 * e], s[2 * e + 1]);
#pragma unroll
        for (int n8 = 1; n8 < kN; ++n8) mx = ptx::max3(mx, s[4 * n8 + 2 * e], s[4 * n8 + 2 * e + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (mx > m[e] + kRescaleLog2) {                 // false while the row is empty
          const float alpha = ptx::ex2(m[e] - mx);      // 0 at the row's first key
          m[e] = mx;
          l[e] *= alpha;
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            o[k][2 * e] *= alpha;
            o[k][2 * e + 1] *= alpha;
          }
        }
        const float sub = m[e] == -INFINITY ? 0.f : m[e];
        float sum = 0.f;
#pragma unroll
        for (int n8 = 0; n8 < kN; ++n8) {
          const float p0 = ptx::ex2(s[4 * n8 + 2 * e] - sub), p1 = ptx::ex2(s[4 * n8 + 2 * e + 1] - sub);
          sum += p0 + p1;
          p[n8 / 2][e + 2 * (n8 & 1)] = ptx::pack2<F16>(p0, p1);
        }
        l[e] += sum;
      }
      {
        const int key = lane & 15, part = lane >> 4;
#pragma unroll
        for (int x = 0; x < kParts; ++x)
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldsm4t(vs + (x * 16 + key) * C::kRowBytes + (((2 * k + part) ^ (key & 7)) << 4), b);
            mma<F16>(o[2 * k], p[x], b[0], b[1]);
            mma<F16>(o[2 * k + 1], p[x], b[2], b[3]);
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
    // the un-normalised output goes to the slot of the warp's last tile, free until its next one:
    // groups of 4 values, their place in a row of D turned by the row against bank conflicts
    if (mine < n) {
      const int last = take == 0 ? C::kStages - 1 : take - 1;
      if (lane == 0) from[warp] = warp * C::kRing + last * C::kStage;
      __syncwarp();                                     // all lanes have read the tile
      uint8_t* const to = smem + warp * C::kRing + last * C::kStage + r0 * D * 4;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const int at4 = ((2 * k + (lane % 4) / 2) ^ r0) * 16 + (lane & 1) * 8;
        *reinterpret_cast<float2*>(to + at4) = make_float2(o[k][0], o[k][1]);
        *reinterpret_cast<float2*>(to + 8 * D * 4 + at4) = make_float2(o[k][2], o[k][3]);
      }
    }
    // what the join needs of this segment; then on to the next one, whose queries travel meanwhile
    const int row0 = seg.block * kRows, n_rows = min(kRows, rows - row0);
    const int64_t qrow = ((int64_t)seg.b * a.H + seg.hk * G) * a.T + row0;
    const bool whole = n == seg.tiles;
    const int seg_s0 = s0, seg_tiles = seg.tiles;
    turn = (turn + n) % kWarps;
    s0 += seg.tiles + kSegment;
    seg.tile = 0;
    if (s0 + kSegment < end) {
      seg.next(a, blocks);
      read_rows();
    }
    __syncthreads();
    for (int x = threadIdx.x; x < n_rows * kQuads; x += kThreads) {
      const int r = x / kQuads, c = x % kQuads * 4;
      float2 ml[kWarps];
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = stat[w * kRows + r];
        mx = fmaxf(mx, ml[w].x);
      }
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // no tile, or none that the row sees.  By the sum, not the maximum: scores that are NaN leave
        // that at -inf, and have to show in the result.
        if (ml[w].y == 0.f) continue;
        const float f = ptx::ex2(ml[w].x - mx);
        const float4 v = *reinterpret_cast<const float4*>(smem + from[w] + r * D * 4 + (((c >> 2) ^ (r & 7)) << 4));
        sum = fmaf(f, ml[w].y, sum);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (!kShared || whole) {
        write_row4<D, F16>(a, qrow + r, c, acc, sum, mx);
      } else {
        const int64_t part = (2 * (int64_t)blockIdx.x + (first_seg ? 0 : 1)) * kRows + r;
        __stcg(reinterpret_cast<float4*>(a.o_part + part * D + c), acc);
        if (c == 0) __stcg(&a.ml_part[part], make_float2(mx, sum));
      }
    }
    const bool was_first = first_seg;
    first_seg = false;
    if (kShared && !whole) {
      // One of several CTAs with tiles of this segment: the one that comes last joins their parts, in
      // the order of the tiles.
      const Shares share(units, n_ctas);
      const int ca = share.owner(seg_s0 + kSegment), cb = share.owner(seg_s0 + kSegment + seg_tiles - 1);
      // the first CTA may have begun inside an earlier segment: this one is then its second part
      const int part0 = 2 * ca + (share.begin(ca) >= seg_s0 ? 0 : 1);
      __syncthreads();
      if (warp == 0) {
        const bool last = all_arrived(a.arrivals, 2 * (int)blockIdx.x + (was_first ? 0 : 1), part0, ca, cb, a.call);
        if (lane == 0) *flag = last ? 1 : 0;
      }
      __syncthreads();
      if (*flag != 0) {
        for (int i = ca + threadIdx.x; i <= cb; i += kThreads) a.arrivals[i == ca ? part0 : 2 * i] = 0ull;
        // Up to kJoin parts at a time: their statistics to shared memory, all in flight together, then
        // their outputs, sixteen in flight, onto what the parts before came to.
        auto part_of = [&](int i) { return (int64_t)(i == ca ? part0 : 2 * i) * kRows; };
        constexpr int kItems = (kRows * kQuads + kThreads - 1) / kThreads;
        float mx[kItems], sum[kItems];
        float4 acc[kItems];
#pragma unroll
        for (int y = 0; y < kItems; ++y) {
          mx[y] = -INFINITY;
          sum[y] = 0.f;
          acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int i0 = ca; i0 <= cb; i0 += C::kJoin) {
          const int np = min(C::kJoin, cb + 1 - i0);
          // sixteen parts' outputs of item x; past the last part its own again, not used
          auto outputs = [&](int x, int i, float4 (&v)[16]) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              v[k] = __ldcg(reinterpret_cast<const float4*>(a.o_part + (part_of(i0 + min(i + k, np - 1)) + x / kQuads) * D +
                                                            x % kQuads * 4));
          };
          float4 v[16];
          if (threadIdx.x < n_rows * kQuads) outputs(threadIdx.x, 0, v);    // under way with the statistics
          __syncthreads();
          for (int x = threadIdx.x; x < np * kRows; x += kThreads)
            joined[x] = __ldcg(&a.ml_part[part_of(i0 + x / kRows) + x % kRows]);
          __syncthreads();
#pragma unroll
          for (int y = 0; y < kItems; ++y) {
            const int x = threadIdx.x + y * kThreads;
            if (x >= n_rows * kQuads) break;
            const int r = x / kQuads;
            float m_new = mx[y];
            for (int i = 0; i < np; ++i) m_new = fmaxf(m_new, joined[i * kRows + r].x);
            // no key of the row so far, and none that is NaN, where the maximum is still -inf
            const float keep = mx[y] == m_new ? 1.f : ptx::ex2(mx[y] - m_new);
            mx[y] = m_new;
            sum[y] *= keep;
            acc[y].x *= keep;
            acc[y].y *= keep;
            acc[y].z *= keep;
            acc[y].w *= keep;
            for (int i = 0; i < np; i += 16) {
              if (y > 0 || i > 0) outputs(x, i, v);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 ml = joined[min(i + k, np - 1) * kRows + r];
                if (i + k >= np || ml.y == 0.f) continue;     // no part, or no key of the row in it
                const float f = ptx::ex2(ml.x - m_new);
                sum[y] = fmaf(f, ml.y, sum[y]);
                acc[y].x = fmaf(f, v[k].x, acc[y].x);
                acc[y].y = fmaf(f, v[k].y, acc[y].y);
                acc[y].z = fmaf(f, v[k].z, acc[y].z);
                acc[y].w = fmaf(f, v[k].w, acc[y].w);
              }
            }
          }
        }
#pragma unroll
        for (int y = 0; y < kItems; ++y) {
          const int x = threadIdx.x + y * kThreads;
          if (x < n_rows * kQuads) write_row4<D, F16>(a, qrow + x / kQuads, x % kQuads * 4, acc[y], sum[y], mx[y]);
        }
      }
    }
    __syncthreads();                                    // the slots and statistics may be written again
  }
  cp_wait<0>();
}

template <int D, bool F16, bool kShared>
cudaError_t launch(const PagedArgs& a, int grid, cudaStream_t s) {
  auto kern = paged_kernel<D, F16, kShared>;
  static LaunchSetup setup;
  const cudaError_t e = prepare_launch(setup, kern, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, Cfg<D>::kSmem, s>>>(a);
  return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t paged(const PagedArgs& a, cudaStream_t s) {
  const int rows = a.H / a.Hkv * a.T;
  const int64_t segments = (int64_t)a.B * a.Hkv * ((rows + kRows - 1) / kRows);
  if (!paged_shares(a.B, a.Hkv, rows, paged_capacity(a.cache), a.ctas)) return launch<D, F16, false>(a, (int)segments, s);
  return launch<D, F16, true>(a, a.ctas, s);
}

}  // namespace

int paged_ctas() {
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess || sms <= 0) sms = 152;      // GB300's when no device can be asked
  return sms * kCtasPerSm;
}

unsigned long long paged_call_number() {
  static std::atomic<unsigned long long> next{
      (unsigned long long)std::chrono::system_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15ull};
  const unsigned long long n = next.fetch_add(1, std::memory_order_relaxed);
  return n != 0 ? n : paged_call_number();             // 0 is a cleared word
}

// Whether CTAs share segments.  Few segments of at most 512 keys get a CTA each, at most two after one
// another in an SM's places: nothing to reckon, nothing to join and no workspace.
bool paged_shares(int B, int Hkv, int rows, int capacity, int ctas) {
  const int64_t segments = (int64_t)B * Hkv * ((rows + kRows - 1) / kRows);
  return capacity > 512 || segments > 2 * (int64_t)ctas;
}

// Whether the units of all segments can be counted in 31 bits.
bool paged_counts(int B, int Hkv, int rows, int capacity) {
  const int64_t segments = (int64_t)B * Hkv * ((rows + kRows - 1) / kRows);
  return segments <= 0x7fffffff / ((int64_t)capacity / 16 + 1 + kSegment);
}

// The workspace: arrivals [2 * ctas], then two parts of 16 rows a CTA, their statistics and outputs.
PagedWorkspace paged_workspace(int ctas, int d) {
  PagedWorkspace w;
  const size_t rows = 2 * (size_t)ctas * kRows;
  w.ml = (2 * (size_t)ctas * sizeof(unsigned long long) + 255) / 256 * 256;
  w.o = w.ml + rows * sizeof(float2);
  w.total = (w.o + rows * d * sizeof(float) + 255) / 256 * 256;
  return w;
}

cudaError_t launch_paged(const PagedArgs& a, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_FP16) return a.d == 64 ? paged<64, true>(a, s) : paged<128, true>(a, s);
  return a.d == 64 ? paged<64, false>(a, s) : paged<128, false>(a, s);
}

}  // namespace fa
