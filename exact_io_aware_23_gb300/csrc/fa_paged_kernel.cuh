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
//
// Chosen pages.  With a list of pages for each (sequence, key head) a segment's tiles run over the
// list's pages in place of the table's; every 16 keys carry their place in the sequence with them.
//
// 8-bit pages.  k_j = ks c_j and v_j = vs e_j, the codes c, e with one scale for each page and head.
// Both kinds of code are whole in fp16 (e4m3: four bits of precision, 2^-9 to 448; int8: whole numbers), so
// the codes become fp16 operands in registers, two to an instruction, and the products are those of fp16
// pages: ks meets the scores of its 16 keys, vs the probabilities.  A bf16 query row is brought into
// fp16's range by a power of two of its own, with its largest value at 2^14: values down to 2^-28 of it
// keep all their bits, smaller ones an absolute error of 2^-39 of it.  The probabilities' products carry vs
// too, and each row has a unit for them, 2^u with u a running maximum of s_ij + log2 vs_j, apart from the
// running maximum of s_ij that goes with the sum l (both raised when a new value exceeds them by more than
// 2^8).  So p vs / 2^u stays below 2^8, and what is rounded below fp16's normal range is off by
// 2^-25 of the row's largest p vs at most: a page of large values that the row gives no weight takes nothing from the
// others.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>

#include <type_traits>

#include "fa_arrivals.cuh"
#include "fa_paged.cuh"
#include "fa_score.cuh"
#include "fa_sm103.cuh"
#include "fa_store.cuh"
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
constexpr int kFlipSegment = 12;           // (4: 10 % longer for 64 chosen pages of 64 keys; 24: the same for d = 64)
// kFlip, d = 128: three CTAs an SM and tiles of 32 keys, at d = 64 four and the same (4 KB in place of 8).
constexpr int flip_ctas(int d) { return d == 128 ? 3 : 4; }
constexpr int kSegment = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kNowhere = 0x7f000000;       // the place of keys that do not exist: behind every row's
constexpr float kRescaleLog2 = 8.0f;       // the running maximum is raised when a score exceeds it by more

// kStore: fa_page_format.  kF16_: the type of 16-bit pages and queries (8-bit pages: of the products).
// kFlip_: keys are the rows of the products and queries their columns (see below).
template <int D_, int kStore_, bool kF16_, bool kPick_, bool kFlip_ = false>
struct Cfg {
  static constexpr int D = D_;
  static constexpr bool k8 = kStore_ != FA_PAGES_16BIT, kInt8 = kStore_ == FA_PAGES_INT8;
  static constexpr bool kFlip = kFlip_;
  static constexpr int kRows = kFlip ? 8 : 16;
  static constexpr bool kDefer = k8;
  static constexpr int kSegment = kFlip ? kFlipSegment : fa::kSegment;
  static constexpr int kCtasPerSm = kFlip ? flip_ctas(D) : fa::kCtasPerSm;
  static constexpr bool kF16 = kF16_ || k8, kPick = kPick_;
  using Elem = std::conditional_t<k8, uint8_t, uint16_t>;
  static constexpr int kElem = sizeof(Elem);
  static constexpr int kRowBytes = D * kElem;
  static constexpr int kKeys = (kFlip && D == 64 ? 2048 : 4096) / kRowBytes;   // keys of a tile: 8 (4) KB with the values
  static constexpr int kParts = kKeys / 16;                   // 16-key parts of a tile, each in one page
  static constexpr int kHalf = kKeys * kRowBytes;             // a tile's keys (or values)
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = 192 * 1024 / kCtasPerSm / (kWarps * kStage);   // 192 KB of tiles an SM
  static constexpr int kRing = kStages * kStage;              // per warp
  static constexpr int kStat = kWarps * kRing;
  static constexpr int kFrom = kStat + kWarps * kRows * 8;
  static constexpr int kParted = kFrom + kWarps * 4 + 16;       // after a flag: statistics to be joined
  static constexpr int kJoin = 64;                              // parts
  // what a tile's parts carry: {ks, vs, place of the first key, -}
  static constexpr int kPending = kParted + kJoin * kRows * 8;  // the CTA's parts of segments
  static constexpr int kMeta = kPending + 64;
  static constexpr int kMetaRing = k8 || kPick ? kStages * kParts * 16 : 0;     // per warp
  static constexpr int kSmem = kMeta + kWarps * kMetaRing;
  static constexpr int kChunks = kRowBytes / 16;              // 16-byte pieces of a row
  static_assert(kStage >= kRows * D * 4, "a warp's output to be joined fits the slot of its last tile");
  // Piece c of row r lies at r * kRowBytes + (c ^ turn(r)) * 16: eight rows' pieces fill all banks.
  static constexpr __host__ __device__ int turn(int r) { return kChunks == 4 ? (r >> 1) & 3 : r & 7; }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;            // 0: the 16 bytes are filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool there) {
  const int n = there ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void st_shared(uint32_t dst, int x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(x) : "memory");
}
__device__ __forceinline__ float4 ld_shared4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
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
// an 8 x 8 matrix of 16-bit values, two adjacent ones of a row to a lane, as its transpose
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

template <typename C>
__host__ __device__ inline int sharing_ctas(int units, int ctas) {
  constexpr int kMinUnits = C::kSegment + kWarps;   // a smaller share costs more in joining than it saves
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

// parts / (parts of a page) by multiplication with the rounded-up reciprocal, exact for the sizes the
// host admits.
__device__ __forceinline__ uint32_t page_of(const PagedArgs& a, uint32_t part) {
  return (uint32_t)(((uint64_t)part * a.parts_magic) >> 36);
}
// The entries of a sequence's lists that count: no more than it has pages.
__device__ __forceinline__ int entries_of(const PagedArgs& a, int len) {
  return min(a.picks, (int)page_of(a, (uint32_t)(len + 15) / 16 + a.page_parts - 1));
}
template <typename C>
__device__ __forceinline__ int tiles_in(const PagedArgs& a, int len) {
  if constexpr (C::kPick) return (entries_of(a, len) * (int)a.page_parts + C::kParts - 1) / C::kParts;
  else return (int)(((uint32_t)len + C::kKeys - 1) / C::kKeys);      // (a length may end within a tile of 2^31)
}
template <typename C>
__device__ __forceinline__ int tiles_of(const PagedArgs& a, int b, int* err) {
  if (new_tokens(a.q_lens, b, a.T) == 0) return 0;
  return tiles_in<C>(a, paged_len(a.cache, b, err));
}
template <typename C>
__device__ __forceinline__ int units_of(const PagedArgs& a, int heads, int b, int* err) {
  const int n = b < a.B ? tiles_of<C>(a, b, err) : 0;
  return n > 0 ? (n + C::kSegment) * heads : 0;
}

// A warp's reckoning of all sequences' units: the first 256 sequences' stay in registers (all their
// lengths are read at once), further ones are read again.
template <typename C>
struct Reckoning {
  int keep[8];
  int total;
  __device__ Reckoning(const PagedArgs& a, int heads, int* err) {
    const int lane = threadIdx.x % 32;
    int sum = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      keep[c] = c * 32 < a.B ? units_of<C>(a, heads, c * 32 + lane, err) : 0;
      sum += keep[c];
    }
    for (int b = 256 + lane; b < a.B; b += 32) sum += units_of<C>(a, heads, b, err);
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
      if (c * 32 < a.B && chunk(keep[c], c * 32)) return;
    for (int b0 = 256; b0 < a.B; b0 += 32)
      if (chunk(units_of<C>(a, heads, b0 + lane, nullptr), b0)) return;
  }
};

// A segment and a tile in it.  The next sequence's lengths are read ahead.
template <typename C>
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
    tiles = count == 0 ? 0 : tiles_in<C>(a, len);
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

// The exponent (biased) by which a bf16 row of this largest value goes to fp16: it becomes that of 2^14;
// infinities and NaN stay what they are.
__device__ __forceinline__ int bf16_exponent(uint32_t bits) { return bits >= 0x7f800000u ? 141 : max((int)(bits >> 23), 15); }

// O = 0 and LSE = -inf for rows [row, row + n)
template <int D>
__device__ __forceinline__ void no_keys(const PagedArgs& a, int64_t row, int n) {
  for (int x = threadIdx.x; x < n * (D / 4); x += kThreads) {
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * D)[x] = make_uint2(0u, 0u);
    if (x < n) a.lse[row + x] = -INFINITY;
  }
}

template <typename C>
__device__ __forceinline__ void write_row4(const PagedArgs& a, int64_t row, int c, float4 acc, float sum, float mx) {
  const float inv = sum != 0.f ? 1.f / sum : 0.f;        // 0: no key; NaN stays
  const bool f16 = C::k8 ? a.f16 != 0 : C::kF16;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * C::D + c) =
      f16 ? make_uint2(ptx::pack2<true>(acc.x * inv, acc.y * inv), ptx::pack2<true>(acc.z * inv, acc.w * inv))
          : make_uint2(ptx::pack2<false>(acc.x * inv, acc.y * inv), ptx::pack2<false>(acc.z * inv, acc.w * inv));
  if (c == 0) a.lse[row] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// A CTA's part of a segment that others have tiles of too.
struct Parted {
  int64_t qrow;                                        // the segment's first query row
  int n_rows;
  int ca, cb;                                          // the CTAs that have tiles of it
  int part0;                                           // the first one's part
};

// Announces this CTA's parts (bits of mine: first, second), and says for a segment that CTAs ca..cb
// share whether all of its parts are there; run by one warp.  Every part has a word of its own, set to the call's number: no atomic
// that 38 CTAs contend for (counting them in one word by compare-and-swap took 18 us at the end of
// B1 H32 Hkv8 with 32K keys).  Between its own store and its reads of the others each CTA has a
// sequentially consistent fence, so the last of them sees all words set, or cleared by one that did;
// should two see them, both join the parts, to the same bits.  Who joins clears the words, for a
// captured call's next run under the same number (another that reads them cleared has nothing left
// to do).  Whatever else a fresh workspace holds is not the number: it has 64 bits, starts at another
// place in every process, and is not used twice in one.  So no launch is spent on clearing the words
// first.  (By cudaMemsetAsync: 3 us of a call's 40.)
__device__ __forceinline__ void announce(unsigned long long* words, int mine, unsigned long long call) {
  const int lane = threadIdx.x % 32;
  if (lane == 0) {
    // releases what the whole CTA wrote before its barrier
    asm volatile("fence.acq_rel.gpu;" ::: "memory");
    if ((mine & 1) != 0) asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(words), "l"(call) : "memory");
    if ((mine & 2) != 0) asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(words + 1), "l"(call) : "memory");
  }
  __syncwarp();
  asm volatile("fence.sc.gpu;" ::: "memory");
}
__device__ __forceinline__ bool all_arrived(unsigned long long* words, int part0, int ca, int cb, unsigned long long call) {
  const int lane = threadIdx.x % 32;
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

// 8-bit pages, whose CTAs announce their parts at the end alone, count them instead, in the word of the
// segment's first part (fa_arrivals.cuh).

// kShared: CTAs share all segments' units.  Otherwise a CTA has one segment to itself (few short
// ones: nothing to join, nothing to reckon).
template <typename C, bool kShared>
__global__ void __launch_bounds__(kThreads, C::kCtasPerSm) paged_kernel(const PagedArgs a) {
  constexpr int D = C::D, kKeys = C::kKeys, kParts = C::kParts, kQuads = D / 4;
  constexpr bool F16 = C::kF16;
  constexpr int kRows = C::kRows;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = a.H / a.Hkv, rows = G * a.T;
  const int blocks = (rows + kRows - 1) / kRows;       // row blocks of a key head
  const int heads = a.Hkv * blocks;

  Walk<C> seg;
  int units = 0, n_ctas = 1, s0 = 0;                   // s0: the segment's first unit
  int begin = 0, end = 0;                              // the CTA's units
  if constexpr (kShared) {
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
      if (tiles_of<C>(a, b, nullptr) == 0) no_keys<D>(a, (int64_t)b * a.H * a.T, a.H * a.T);
    const Reckoning<C> all(a, heads, blockIdx.x == 0 && warp == 0 ? a.err : nullptr);
    units = all.total;
    n_ctas = sharing_ctas<C>(units, gridDim.x);
    if ((int)blockIdx.x >= n_ctas || units == 0) return;
    const Shares share(units, n_ctas);
    begin = share.begin(blockIdx.x);
    end = share.begin(blockIdx.x + 1);
    int b, before;
    all.find(a, heads, begin, &b, &before);
    seg.start(a, b);
    const int hr = (begin - before) / (seg.tiles + C::kSegment);
    seg.hk = hr / blocks;
    seg.block = hr % blocks;
    s0 = before + hr * (seg.tiles + C::kSegment);
    seg.tile = max(0, begin - s0 - C::kSegment);
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
    end = seg.tiles + C::kSegment;
  }
  // tiles of the current segment up to this number are the CTA's
  auto last_tile = [&](int first_unit, int tiles) { return min(tiles, end - first_unit - C::kSegment); };

  // ---- the warp's copies: every fourth tile of the CTA's, into its own ring ----------------------
  const uint32_t ring = ptx::smem_u32(smem) + warp * C::kRing;
  Walk<C> load = seg;
  int load_s0 = s0;
  bool more = true;
  auto step = [&](int n) {                              // n tiles on
    int t = load.tile + n;
    while (t >= load.tiles) {
      t -= load.tiles;
      load_s0 += load.tiles + C::kSegment;
      load.next(a, blocks);
      if (load_s0 + C::kSegment >= end) break;
    }
    load.tile = t;
    more = load_s0 + C::kSegment + t < end;
  };
  // The next tile's parts of 16 keys: their pages, and their first rows in them.
  int page[kParts], first[kParts];
  // Chosen pages: also their number in the sequence (-1: none).  The lanes keep 32 entries of a list, from
  // number `held` of segment `held_s0` on, so that the two reads on the way to a page, one after
  // another, are waited for once in 32 pages.
  int number[C::kPick ? kParts : 1], held = 0, held_s0 = -1, lane_number = -1, lane_page = 0;
  auto read_pages = [&]() {
    if (!more) return;
    const int32_t* row = a.cache.table + load.b * a.cache.table_stride;
    if constexpr (C::kPick) {
      const int e0 = page_of(a, load.tile * kParts), e1 = page_of(a, load.tile * kParts + kParts - 1);
      if (held_s0 != load_s0 || e1 >= held + 32) {
        held_s0 = load_s0;
        held = e0;
        const int n = entries_of(a, load.len), i = e0 + lane;
        lane_number = i < n ? a.pages[((int64_t)load.b * a.Hkv + load.hk) * a.picks + i] : -1;
        const bool there = lane_number >= 0 && lane_number < (int)page_of(a, (uint32_t)(load.len + 15) / 16 + a.page_parts - 1);
        lane_number = there ? lane_number : -1;
        lane_page = there ? row[lane_number] : 0;
      }
    }
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
      const uint32_t part = load.tile * kParts + x;
      const uint32_t at = page_of(a, part);
      first[x] = (int)(part - at * a.page_parts) * 16;
      if constexpr (C::kPick) {
        number[x] = __shfl_sync(0xffffffffu, lane_number, (int)at - held);
        page[x] = __shfl_sync(0xffffffffu, lane_page, (int)at - held);
      } else {
        page[x] = x == 0 || (int)part * 16 < load.len ? row[at] : 0;
      }
    }
  };
  more = s0 + C::kSegment + seg.tile < end;
  if (more) step(warp);
  read_pages();
  // This lane's 16-byte pieces: column c of rows row, row + kStep, ...
  using Elem = typename C::Elem;
  constexpr int kChunks = C::kChunks, kStep = 32 / kChunks;
  const int lane_row = lane / kChunks, lane_col = lane % kChunks;
  const uint32_t lane_off = lane_row * C::kRowBytes + ((lane_col ^ C::turn(lane_row)) << 4);
  const Elem* const kbase = static_cast<const Elem*>(a.cache.k) + lane_col * (16 / C::kElem);
  const int64_t v_off = static_cast<const Elem*>(a.cache.v) - static_cast<const Elem*>(a.cache.k);
  const uint32_t metas = ptx::smem_u32(smem) + C::kMeta + warp * C::kMetaRing;
  const int64_t row_step = kStep * a.cache.token_stride;
  int slot = 0;
  auto copy_tile = [&]() {
    if (more) {
      const uint32_t dst = ring + slot * C::kStage + lane_off;
#pragma unroll
      for (int x = 0; x < kParts; ++x) {
        int n = load.len - (load.tile * kParts + x) * 16;      // keys of the part that exist
        if constexpr (C::kPick) n = number[x] < 0 ? 0 : load.len - number[x] * a.cache.page_size - first[x];
        if ((unsigned)page[x] >= (unsigned)a.cache.n_pages && n > 0) {
          if (lane == 0) atomicExch(a.err, kDevBadOffsets);    // reported, not followed
          n = 0;
        }
        if constexpr (C::k8 || C::kPick) {
          const uint32_t to = metas + (slot * kParts + x) * 16;
          if constexpr (C::k8) {
            if (lane < 2) {
              const float* scales = lane == 0 ? a.k_scales : a.v_scales;
              cp4(to + lane * 4, scales + (n > 0 ? (int64_t)page[x] * a.Hkv + load.hk : 0), n > 0);
            }
          }
          if constexpr (C::kPick) {
            // no key there: a place that no row sees
            if (lane == 2) st_shared(to + 8, n > 0 ? number[x] * a.cache.page_size + first[x] : kNowhere);
          }
        }
        const Elem* src = kbase;
        if (n > 0)
          src += page[x] * a.cache.page_stride + load.hk * a.cache.head_stride + (first[x] + lane_row) * a.cache.token_stride;
        if (n >= 16) {
#pragma unroll
          for (int i = 0; i < 16 / kStep; ++i, src += row_step) {
            const uint32_t to = (dst ^ (C::turn(i * kStep) << 4)) + (x * 16 + i * kStep) * C::kRowBytes;
            cp16(to, src);
            cp16(to + C::kHalf, src + v_off);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16 / kStep; ++i, src += row_step) {
            const bool there = i * kStep + lane_row < n;
            const Elem* from = there ? src : kbase;
            const uint32_t to = (dst ^ (C::turn(i * kStep) << 4)) + (x * 16 + i * kStep) * C::kRowBytes;
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
  Parted* const parted = reinterpret_cast<Parted*>(smem + C::kPending);
  if (threadIdx.x == 0) *flag = 0;
  int take = 0;                                         // ring slot of the next tile
  int turn = 0;                                         // the warp whose turn the segment's first tile is
  bool first_seg = true;

  // the segment's queries as mma operands; per row its slope and the keys it sees
  constexpr bool kFlip = C::kFlip;
  uint32_t q[D / 16][kFlip ? 2 : 4];
  int limit[2], full;
  float slope[2];
  float unit_q[2];                                      // 8-bit pages: what the operand's values count
  auto read_rows = [&]() {
    const int row0 = seg.block * kRows, n_rows = min(kRows, rows - row0);
    const int64_t qrow = ((int64_t)seg.b * a.H + seg.hk * G) * a.T + row0;
    if constexpr (!C::k8) {
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + qrow * D + r0 * D + c0);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[i][e] = r0 + (e & 1) * 8 < n_rows ? __ldg(qp + ((e & 1) * 8 * D + i * 16 + (e >> 1) * 8) / 2) : 0u;
    } else if constexpr (kFlip) {
      // the lane's values are row r0's, its scores those of rows c0 and c0 + 1
      const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (qrow + r0) * D + 2 * c0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint2 v = r0 < n_rows ? __ldg(reinterpret_cast<const uint2*>(qp + i * 16)) : make_uint2(0u, 0u);
        q[i][0] = v.x;
        q[i][1] = v.y;
      }
    } else {
      // four adjacent codes of a key are a register: the products' columns 2 i, 2 i + 1 and 2 i + 8, 2 i + 9 of
      // lane i are values 4 i to 4 i + 3 of the 16
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + qrow * D + r0 * D + 2 * c0);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint2 v = r0 + e * 8 < n_rows ? __ldg(reinterpret_cast<const uint2*>(qp + (e * 8 * D + i * 16) / 2)) : make_uint2(0u, 0u);
          q[i][e] = v.x;
          q[i][e + 2] = v.y;
        }
    }
    full = 0x7fffffff;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + (kFlip ? c0 + e : r0 + e * 8);
      const int h = a.T == 1 ? r : r / a.T, t = r - h * a.T;
      limit[e] = r < rows && t < seg.count ? seg.len - seg.count + t + 1 : 0;
      if (r < rows) full = min(full, limit[e]);
      slope[e] = a.score.slopes != nullptr && r < rows ? __ldg(a.score.slopes + seg.hk * G + h) * kLog2e : 0.f;
    }
    full = __reduce_min_sync(0xffffffffu, full);        // keys that every row sees
  };
  // 8-bit pages: bf16 queries as fp16 in units of their own (once they are there)
  auto convert_rows = [&]() {
    if constexpr (!C::k8) return;
    unit_q[0] = unit_q[1] = 1.f;
    if (a.f16) return;
    if constexpr (kFlip) {
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w) mx = max(mx, max(q[i][w] << 16 & 0x7fff0000u, q[i][w] & 0x7fff0000u));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int x = bf16_exponent(mx);
      const float f = __uint_as_float((uint32_t)(268 - x) << 23), unit = __uint_as_float((uint32_t)(x - 14) << 23);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w)
          q[i][w] = ptx::pack_f16(__uint_as_float(q[i][w] << 16) * f, __uint_as_float(q[i][w] & 0xffff0000u) * f);
#pragma unroll
      for (int e = 0; e < 2; ++e) unit_q[e] = __shfl_sync(0xffffffffu, unit, 4 * (c0 + e));
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int w = e; w < 4; w += 2) mx = max(mx, max(q[i][w] << 16 & 0x7fff0000u, q[i][w] & 0x7fff0000u));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int x = bf16_exponent(mx);
        const float f = __uint_as_float((uint32_t)(268 - x) << 23);      // 2^(141 - x)
        unit_q[e] = __uint_as_float((uint32_t)(x - 14) << 23);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int w = e; w < 4; w += 2)
            q[i][w] = ptx::pack_f16(__uint_as_float(q[i][w] << 16) * f, __uint_as_float(q[i][w] & 0xffff0000u) * f);
      }
    }
  };
  // Who else has tiles of the segment, worked out while its first ones are on their way.
  auto note_parted = [&](int k) {
    const int last = last_tile(s0, seg.tiles);
    if (!kShared || threadIdx.x != 0 || last <= seg.tile || (seg.tile == 0 && last == seg.tiles)) return;
    const Shares share(units, n_ctas);
    const int ca = share.owner(s0 + C::kSegment), cb = share.owner(s0 + C::kSegment + seg.tiles - 1);
    const int row0 = seg.block * kRows;
    // the first CTA may have begun inside an earlier segment: this one is then its second part
    const int part0 = 2 * ca + (share.begin(ca) >= s0 ? 0 : 1);
    parted[k] = Parted{((int64_t)seg.b * a.H + seg.hk * G) * a.T + row0, min(kRows, rows - row0), ca, cb, part0};
    if (C::kDefer) open_count(a.arrivals + part0, a.call);
  };
  read_rows();                                          // before the copies fill the way to memory
#pragma unroll 1
  for (int i = 0; i < C::kStages - 1; ++i) copy_tile();
  convert_rows();
  note_parted(0);

  // Segments that other CTAs have tiles of too, the CTA's first one and its last: the CTA that comes last
  // joins their parts, in the order of the tiles.  With 8-bit pages both are announced together, at the end:
  // done where the first one ends, it held its CTA up by 9 us (B2 H32 Hkv8 d128 with 100K e4m3 keys).
  // With 16-bit ones each is done with at its end, while twice the bytes are on their way: no CTA then
  // has two segments to join at the end (B64, 1 to 8192 keys, 159 us against 163).
  auto finish = [&](const int mine) {                   // bits: the first part, the second
    if (C::kDefer) {
      if (threadIdx.x == 0) {
        asm volatile("fence.acq_rel.gpu;" ::: "memory");  // releases what the whole CTA wrote before its barrier
        int there = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if ((mine >> k & 1) != 0 && count_part(a.arrivals + parted[k].part0, parted[k].cb - parted[k].ca + 1)) there |= 1 << k;
        if (there != 0) asm volatile("fence.acq_rel.gpu;" ::: "memory");     // the parts, for the CTA after its barrier
        *flag = there;
      }
    } else if (warp == 0) {
      announce(a.arrivals + 2 * blockIdx.x, mine, a.call);
      int there = 0;
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        if ((mine >> k & 1) == 0) continue;
        if (all_arrived(a.arrivals, parted[k].part0, parted[k].ca, parted[k].cb, a.call)) there |= 1 << k;
      }
      if (lane == 0) *flag = there;
    }
    __syncthreads();
    const int last = *flag;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      if ((last >> k & 1) == 0) continue;
      const int n_rows = parted[k].n_rows;
      const int64_t qrow = parted[k].qrow;
      const int ca = parted[k].ca, cb = parted[k].cb, part0 = parted[k].part0;
      if (C::kDefer) {
        if (threadIdx.x == 0) a.arrivals[part0] = 0ull;
      } else {
        for (int i = ca + threadIdx.x; i <= cb; i += kThreads) a.arrivals[i == ca ? part0 : 2 * i] = 0ull;
      }
      // Up to kJoin parts at a time: their statistics to shared memory, all in flight together, then
      // their outputs, several in flight, onto what the parts before came to.
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
        // several parts' outputs of item x; past the last part its own again, not used
        constexpr int kFlight = 16;
        auto outputs = [&](int x, int i, float4 (&v)[kFlight]) {
#pragma unroll
          for (int k = 0; k < kFlight; ++k)
            v[k] = __ldcg(reinterpret_cast<const float4*>(a.o_part + (part_of(i0 + min(i + k, np - 1)) + x / kQuads) * D +
                                                          x % kQuads * 4));
        };
        float4 v[kFlight];
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
          for (int i = 0; i < np; i += kFlight) {
            if (y > 0 || i > 0) outputs(x, i, v);
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
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
        if (x < n_rows * kQuads) write_row4<C>(a, qrow + x / kQuads, x % kQuads * 4, acc[y], sum[y], mx[y]);
      }
    }
  };

#pragma unroll 1
  while (s0 + C::kSegment < end) {
    const int n = last_tile(s0, seg.tiles) - seg.tile;  // the CTA's tiles of the segment: at least one
    const int mine = (warp - turn + kWarps) % kWarps;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float u[2] = {-FLT_MAX, -FLT_MAX};                  // 8-bit pages: what the output counts, a power of two's exponent
    // kFlip: o[j] are values 16 j + 2 r0 and the next one of rows c0 and c0 + 1
    constexpr int kOut = kFlip ? D / 16 : D / 8;
    float o[kOut][4];
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll 1
    for (int i = mine; i < n; i += kWarps) {
      cp_wait<C::kStages - 2>();
      __syncwarp();                                   // this tile is there, the last one read
      copy_tile();                                    // into the last one's slot
      const uint32_t ks = ring + take * C::kStage, vs = ks + C::kHalf;
      float4 meta[C::kMetaRing > 0 ? kParts : 1];
      if constexpr (C::kMetaRing > 0) {
#pragma unroll
        for (int x = 0; x < kParts; ++x) meta[x] = ld_shared4(metas + (take * kParts + x) * 16);
      }
      take = take + 1 == C::kStages ? 0 : take + 1;
      constexpr int kN = kKeys / 8;                     // groups of 8 keys
      constexpr int kScores = kFlip ? kKeys / 4 : kKeys / 2;
      // row r0: s[4 n], s[4 n + 1] of key group n; r0 + 8: the next two.
      // kFlip: s[2 n], s[2 n + 1]: key r0 of group n, rows c0 and c0 + 1
      float s[kScores];
#pragma unroll
      for (int e = 0; e < kScores; ++e) s[e] = 0.f;
      // score e: its key's place in the tile without the lane's part, and which of the lane's two rows
      auto key_of = [](int e) { return kFlip ? (e >> 1) * 8 : (e >> 2) * 8 + (e & 1); };
      auto row_of = [](int e) { return kFlip ? e & 1 : (e >> 1) & 1; };
      const int lane_key = kFlip ? r0 : c0;
      if constexpr (kFlip) {
        float odd[kScores];                             // the other half of the products, for shorter chains
#pragma unroll
        for (int e = 0; e < kScores; ++e) odd[e] = 0.f;
        const int key = (lane & 7) + ((lane >> 4) << 3), part = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < kChunks / 2; ++k)
#pragma unroll
          for (int x = 0; x < kParts; ++x) {
            uint32_t b[4];
            ldsm4(ks + (x * 16 + key) * C::kRowBytes + (((2 * k + part) ^ C::turn(key)) << 4), b);
            uint32_t lhs[4];
            codes<C::kInt8, false>(b[0], lhs[0], lhs[2]);
            codes<C::kInt8, false>(b[2], lhs[1], lhs[3]);
            mma<F16>(&s[4 * x], lhs, q[2 * k][0], q[2 * k][1]);
            codes<C::kInt8, false>(b[1], lhs[0], lhs[2]);
            codes<C::kInt8, false>(b[3], lhs[1], lhs[3]);
            mma<F16>(&odd[4 * x], lhs, q[2 * k + 1][0], q[2 * k + 1][1]);
          }
#pragma unroll
        for (int e = 0; e < kScores; ++e) s[e] += odd[e];
      } else {
        // matrices of a load: keys 0-7 and 8-15, two groups of 8 values each
        const int key = (lane & 7) + ((lane >> 4) << 3), part = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < kChunks / 2; ++k)
#pragma unroll
          for (int x = 0; x < kParts; ++x) {
            uint32_t b[4];
            ldsm4(ks + (x * 16 + key) * C::kRowBytes + (((2 * k + part) ^ C::turn(key)) << 4), b);
            if constexpr (!C::k8) {
              mma<F16>(&s[8 * x], q[k], b[0], b[1]);
              mma<F16>(&s[8 * x + 4], q[k], b[2], b[3]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {             // keys 0-7 and 8-15, two pieces of 16 values each
                uint32_t lo, hi;
                codes<C::kInt8, false>(b[e], lo, hi);
                mma<F16>(&s[8 * x + 4 * (e >> 1)], q[2 * k + (e & 1)], lo, hi);
              }
            }
          }
      }
      // scores in the log2 domain
      int key0[kParts];
      bool hidden = false;                              // some row does not see all of the tile
#pragma unroll
      for (int x = 0; x < kParts; ++x) {
        key0[x] = C::kPick ? __float_as_int(meta[x].z) : (seg.tile + i) * kKeys + x * 16;
        hidden = hidden || key0[x] > full - 16;
      }
      if constexpr (C::k8) {
        const float c = a.score.cap_log2 == 0.f ? c_log2 : 1.f;
#pragma unroll
        for (int e = 0; e < kScores; ++e) s[e] *= meta[key_of(e) / 16].x * c * unit_q[row_of(e)];
      }
      if (a.score.cap_log2 == 0.f) {
        if constexpr (!C::k8) {
#pragma unroll
          for (int e = 0; e < kScores; ++e) s[e] *= c_log2;
        }
      } else if (poly_fits(s, a.score.poly_limit)) {
#pragma unroll
        for (int e = 0; e < kScores; e += 2) {
          const float2 t = tanh_poly(make_float2(s[e], s[e + 1]), a.score);
          s[e] = t.x * a.score.cap_log2;
          s[e + 1] = t.y * a.score.cap_log2;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kScores; ++e) s[e] = a.score.cap_log2 * tanh_one(s[e], a.score);
      }
      if (a.score.slopes != nullptr) {
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
          float ahead[2];                               // minus the distance at the lane's first key, exact
#pragma unroll
          for (int e = 0; e < 2; ++e) ahead[e] = (float)(key0[C::kPick ? x : 0] + lane_key - (limit[e] - 1));
#pragma unroll
          for (int e = x * kScores / kParts; e < (x + 1) * kScores / kParts; ++e)
            s[e] = fmaf(slope[row_of(e)], ahead[row_of(e)] + (float)(key_of(e) - (C::kPick ? 16 * x : 0)), s[e]);
        }
      }
      auto sees = [&](int e) { return key0[key_of(e) / 16] + key_of(e) % 16 + lane_key < limit[row_of(e)]; };
      if (hidden) {
#pragma unroll
        for (int e = 0; e < kScores; ++e) s[e] = sees(e) ? s[e] : -INFINITY;
      }
      // 8-bit pages: the largest of each row's scores with their values' scales raises the row's unit; then, of the
      // keys of each part, by how much a probability counts in it
      float gain[C::k8 ? kParts : 1][2], top[2] = {-INFINITY, -INFINITY};
      auto raise_units = [&]() {
        float w[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
          const float lg = __log2f(meta[x].y);          // (NaN raises nothing)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = -INFINITY;
#pragma unroll
            for (int i = x * kScores / kParts; i < (x + 1) * kScores / kParts; ++i)
              if (row_of(i) == e) t = fmaxf(t, s[i]);
            top[e] = fmaxf(top[e], t);
            w[e] = fmaxf(w[e], t + lg);
          }
        }
        if (!__any_sync(0xffffffffu, w[0] > u[0] + kRescaleLog2 || w[1] > u[1] + kRescaleLog2)) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = kFlip ? 4 : 1; d < (kFlip ? 32 : 4); d <<= 1) w[e] = fmaxf(w[e], __shfl_xor_sync(0xffffffffu, w[e], d));
          if (w[e] > u[e] + kRescaleLog2) {
            const float beta = ptx::ex2(u[e] - w[e]);
            u[e] = w[e];
#pragma unroll
            for (int k = 0; k < kOut; ++k)
#pragma unroll
              for (int i = 0; i < 2; ++i) o[k][kFlip ? e + 2 * i : 2 * e + i] *= beta;
          }
        }
      };
      auto set_gains = [&]() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // (far above where the largest score is one of values that are next to nothing)
          const float r = ptx::ex2(fminf(m[e] - u[e], 126.f));
#pragma unroll
          for (int x = 0; x < kParts; ++x) gain[x][e] = ptx::min_nan(meta[x].y * r, 0x1p120f);   // finite, for probabilities that are 0
        }
      };
      if constexpr (C::k8) raise_units();
      if constexpr (kFlip) {
        uint32_t p[kN];                                 // the keys of group n, transposed: right operands
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = top[e];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          if (mx > m[e] + kRescaleLog2) {               // false while the row is empty
            const float alpha = ptx::ex2(m[e] - mx);    // 0 at the row's first key
            m[e] = mx;
            l[e] *= alpha;
          }
          const float sub = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
          for (int n8 = 0; n8 < kN; ++n8) s[2 * n8 + e] = ptx::ex2(s[2 * n8 + e] - sub);
#pragma unroll
          for (int n8 = 0; n8 < kN; n8 += 2) l[e] += s[2 * n8 + e] + s[2 * n8 + 2 + e];
        }
        set_gains();
#pragma unroll
        for (int n8 = 0; n8 < kN; ++n8) {
          // a scale that is NaN meets the keys that the row sees, all of them, and no others
          const float* const f = gain[n8 / 2];
          const float f0 = hidden && !sees(2 * n8) ? 0.f : f[0], f1 = hidden && !sees(2 * n8 + 1) ? 0.f : f[1];
          p[n8] = transposed(ptx::pack2<F16>(s[2 * n8] * f0, s[2 * n8 + 1] * f1));
        }
        const int key = lane & 15, part = lane >> 4;
#pragma unroll
        for (int x = 0; x < kParts; ++x)
#pragma unroll
          for (int k = 0; k < kChunks / 2; ++k) {
            uint32_t b[4];
            ldsm4t(vs + (x * 16 + key) * C::kRowBytes + (((2 * k + part) ^ C::turn(key)) << 4), b);
            // a register holds values 2 i, 2 i + 1 of two keys: the even ones are the product's upper rows, the
            // odd ones its lower
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t lhs[4];
              codes<C::kInt8, true>(b[2 * e], lhs[0], lhs[1]);
              codes<C::kInt8, true>(b[2 * e + 1], lhs[2], lhs[3]);
              mma<F16>(o[2 * k + e], lhs, p[2 * x], p[2 * x + 1]);
            }
          }
      } else {
      uint32_t p[kParts][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = top[e];
        if constexpr (!C::k8) {
          mx = fmaxf(s[2 * e], s[2 * e + 1]);
#pragma unroll
          for (int n8 = 1; n8 < kN; ++n8) mx = ptx::max3(mx, s[4 * n8 + 2 * e], s[4 * n8 + 2 * e + 1]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (mx > m[e] + kRescaleLog2) {                 // false while the row is empty
          const float alpha = ptx::ex2(m[e] - mx);      // 0 at the row's first key
          m[e] = mx;
          l[e] *= alpha;
          if constexpr (!C::k8) {
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
              o[k][2 * e] *= alpha;
              o[k][2 * e + 1] *= alpha;
            }
          }
        }
        const float sub = m[e] == -INFINITY ? 0.f : m[e];
        float sum = 0.f;
#pragma unroll
        for (int n8 = 0; n8 < kN; ++n8) {
          const float p0 = ptx::ex2(s[4 * n8 + 2 * e] - sub), p1 = ptx::ex2(s[4 * n8 + 2 * e + 1] - sub);
          sum += p0 + p1;
          if constexpr (C::k8) {
            s[4 * n8 + 2 * e] = p0;
            s[4 * n8 + 2 * e + 1] = p1;
          } else {
            p[n8 / 2][e + 2 * (n8 & 1)] = ptx::pack2<F16>(p0, p1);
          }
        }
        l[e] += sum;
      }
      if constexpr (C::k8) {
        set_gains();
#pragma unroll
        for (int n8 = 0; n8 < kN; ++n8)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // a scale that is NaN meets the keys that the row sees, all of them, and no others
            const int i = 4 * n8 + 2 * e;
            const float f = gain[n8 / 2][e], f0 = hidden && !sees(i) ? 0.f : f, f1 = hidden && !sees(i + 1) ? 0.f : f;
            p[n8 / 2][e + 2 * (n8 & 1)] = ptx::pack2<F16>(s[i] * f0, s[i + 1] * f1);
          }
      }
      {
        const int key = lane & 15, part = lane >> 4;
#pragma unroll
        for (int x = 0; x < kParts; ++x)
#pragma unroll
          for (int k = 0; k < kChunks / 2; ++k) {
            uint32_t b[4];
            ldsm4t(vs + (x * 16 + key) * C::kRowBytes + (((2 * k + part) ^ C::turn(key)) << 4), b);
            if constexpr (!C::k8) {
              mma<F16>(o[2 * k], p[x], b[0], b[1]);
              mma<F16>(o[2 * k + 1], p[x], b[2], b[3]);
            } else {
              // a register holds values 2 i, 2 i + 1 of two keys: even and odd values are products of their own
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t even[2], odd[2];
                codes<C::kInt8, true>(b[2 * e], even[0], odd[0]);
                codes<C::kInt8, true>(b[2 * e + 1], even[1], odd[1]);
                mma<F16>(o[4 * k + 2 * e], p[x], even[0], even[1]);
                mma<F16>(o[4 * k + 2 * e + 1], p[x], odd[0], odd[1]);
              }
            }
          }
      }
    }
    }
    // ---- the segment's end: join the warps -------------------------------------------------------
    if constexpr (kFlip) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
        if (lane < 4) stat[warp * kRows + c0 + e] = make_float2(m[e], l[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      }
      if (lane % 4 == 0) {
        stat[warp * kRows + r0] = make_float2(m[0], l[0]);
        stat[warp * kRows + r0 + 8] = make_float2(m[1], l[1]);
      }
    }
    // the un-normalised output goes to the slot of the warp's last tile, free until its next one:
    // groups of 4 values, their place in a row of D turned by the row against bank conflicts
    if (mine < n) {
      // 8-bit pages: a row's output, from its unit to the one that goes with its maximum
      float unit_o[2] = {1.f, 1.f};
      if constexpr (C::k8) {
#pragma unroll
        for (int e = 0; e < 2; ++e) unit_o[e] = m[e] == -INFINITY ? 1.f : ptx::ex2(u[e] - m[e]);
      }
      const int last = take == 0 ? C::kStages - 1 : take - 1;
      if (lane == 0) from[warp] = warp * C::kRing + last * C::kStage;
      __syncwarp();                                     // all lanes have read the tile
      uint8_t* const to = smem + warp * C::kRing + last * C::kStage + (kFlip ? c0 : r0) * D * 4;
      if constexpr (kFlip) {
#pragma unroll
        for (int j = 0; j < kOut; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(to + e * D * 4 + ((4 * j + r0 / 2) ^ (c0 + e)) * 16 + (r0 & 1) * 8) =
                make_float2(o[j][e] * unit_o[e], o[j][2 + e] * unit_o[e]);
      } else if constexpr (!C::k8) {
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const int at4 = ((2 * k + (lane % 4) / 2) ^ r0) * 16 + (lane & 1) * 8;
          *reinterpret_cast<float2*>(to + at4) = make_float2(o[k][0], o[k][1]);
          *reinterpret_cast<float2*>(to + 8 * D * 4 + at4) = make_float2(o[k][2], o[k][3]);
        }
      } else {
        // columns 2 i, 2 i + 1 of the even and the odd products are values 4 i to 4 i + 3 of 16
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const int at4 = ((4 * j + lane % 4) ^ r0) * 16;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(to + e * 8 * D * 4 + at4) =
                make_float4(o[2 * j][2 * e] * unit_o[e], o[2 * j + 1][2 * e] * unit_o[e], o[2 * j][2 * e + 1] * unit_o[e],
                            o[2 * j + 1][2 * e + 1] * unit_o[e]);
        }
      }
    }
    // what the join needs of this segment; then on to the next one, whose queries travel meanwhile
    const int row0 = seg.block * kRows, n_rows = min(kRows, rows - row0);
    const int64_t qrow = ((int64_t)seg.b * a.H + seg.hk * G) * a.T + row0;
    const bool whole = n == seg.tiles;
    turn = (turn + n) % kWarps;
    s0 += seg.tiles + C::kSegment;
    seg.tile = 0;
    if (s0 + C::kSegment < end) {
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
        write_row4<C>(a, qrow + r, c, acc, sum, mx);
      } else {
        const int64_t part = (2 * (int64_t)blockIdx.x + (first_seg ? 0 : 1)) * kRows + r;
        __stcg(reinterpret_cast<float4*>(a.o_part + part * D + c), acc);
        if (c == 0) __stcg(&a.ml_part[part], make_float2(mx, sum));
      }
    }
    if (kShared && C::kDefer && !whole && threadIdx.x == 0) *flag |= first_seg ? 1 : 2;
    const bool was_first = first_seg;
    first_seg = false;
    if (s0 + C::kSegment < end) convert_rows();
    __syncthreads();                                    // the slots and statistics may be written again
    if constexpr (kShared && !C::kDefer)
      if (!whole) finish(was_first ? 1 : 2);
    if (s0 + C::kSegment < end) note_parted(1);
  }
  cp_wait<0>();
  if constexpr (kShared && C::kDefer) {
    __syncthreads();                                    // (a CTA may have had units, but no tile)
    const int mine = *flag;
    __syncthreads();                                    // the word is written again
    if (mine != 0) finish(mine);
  }
}

template <typename C, bool kShared>
cudaError_t launch(const PagedArgs& a, int grid, cudaStream_t s) {
  auto kern = paged_kernel<C, kShared>;
  static LaunchSetup setup;
  const cudaError_t e = prepare_launch(setup, kern, C::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, C::kSmem, s>>>(a);
  return cudaGetLastError();
}

template <typename C>
cudaError_t paged(const PagedArgs& a, cudaStream_t s) {
  const int rows = a.H / a.Hkv * a.T;
  const int64_t segments = (int64_t)a.B * a.Hkv * ((rows + C::kRows - 1) / C::kRows);
  if (!paged_shares(a.B, a.Hkv, rows, paged_span(a), a.ctas)) return launch<C, false>(a, (int)segments, s);
  return launch<C, true>(a, a.ctas, s);
}

// 8-bit pages: up to 8 rows of a group as columns of the products.
template <int D, int kStore, bool kPick>
cudaError_t paged8(const PagedArgs& a, cudaStream_t s) {
  if (a.H / a.Hkv * a.T > 8) return paged<Cfg<D, kStore, true, kPick>>(a, s);
  PagedArgs f = a;
  f.ctas = a.ctas / kCtasPerSm * flip_ctas(D);
  return paged<Cfg<D, kStore, true, kPick, true>>(f, s);
}
template <int kStore>
cudaError_t paged8(const PagedArgs& a, cudaStream_t s) {
  if (a.pages != nullptr) return a.d == 64 ? paged8<64, kStore, true>(a, s) : paged8<128, kStore, true>(a, s);
  return a.d == 64 ? paged8<64, kStore, false>(a, s) : paged8<128, kStore, false>(a, s);
}

}  // namespace
}  // namespace fa
