// Pages for sequences that grow and shrink: block tables, free pages and the places of new tokens, from
// the lengths alone, all on the device.
//
// With held = ceil(old / page) and want = ceil(new / page), G and R the sums of the growths and of the
// releases of the sequences before b, and the free pages a ring of n from `first` on, `count` of them:
//     b grows:    table[b][held + j] = ring[(first + G_b + j) mod n]
//     b shrinks:  ring[(first + count + R_b + j) mod n] = table[b][want + j]
//     slot of its token at place p:  table[b][p / page] * page + p % page
// Pages given back join the ring's end and are not handed out in the same call, so every place is read or
// written once and nothing waits for another's result: each thread finds a new token's page from the sums
// alone, whether the table has it already or not.
//
// What bounds it: the latency of a launch and of three reads one after another (lengths, state, ring), then the
// bytes of the slots.  Few tokens: one block does it all.  Many: blocks of their own place 2048 tokens each, after
// summing up the lengths for themselves, while the first one sees to the tables: nothing that it writes is
// read by them, unless the caller has the lengths or the state written over its inputs, and then it runs
// behind them as a second launch.  (40 sequences of up to 4096 tokens: 27 us by a cluster of 8 blocks with a
// barrier before the lengths are written, 12 in two launches, 9 in one.)
#include <cuda_runtime.h>

#include "fa_paged.cuh"
#include "fa_sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kPlaceTokens = 2048;         // a block's that places tokens of a sequence

// The pages of n tokens, by multiplication with the page size's rounded-up reciprocal: exact for n below 2^31 and
// pages of up to 4096 tokens (2^43 / page, the error below n / 2^43 of a page).
__device__ __forceinline__ int whole_pages(const AssignArgs& a, int n) { return (int)__umul64hi((uint64_t)(uint32_t)n << 21, a.page_magic); }
__device__ __forceinline__ int pages_for(const AssignArgs& a, int n) {
  const int w = whole_pages(a, n);
  return w + (n - w * a.page_size > 0 ? 1 : 0);
}

struct Change {
  int old, now, held, want;
};
__device__ __forceinline__ Change change_of(const AssignArgs& a, int b) {
  Change c;
  c.old = a.old_lens[b];
  c.now = a.new_lens[b];
  c.held = pages_for(a, max(c.old, 0));
  c.want = pages_for(a, max(c.now, 0));
  return c;
}

// What the whole call comes to; the same in every block.
struct Totals {
  int64_t grow, less, grow_before;         // the last: of the sequences before `upto`
  bool ok;
};
template <int kThr>
__device__ __forceinline__ Totals totals_of(const AssignArgs& a, int first, int count, int upto, int64_t (*words)[kThr / 32]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  // growth (with a large number for a length that is none), releases, growth before
  int64_t x[3] = {0, 0, 0};
  for (int b = threadIdx.x; b < a.B; b += kThr) {
    const Change c = change_of(a, b);
    const int grow = max(c.want - c.held, 0);
    x[0] += c.old < 0 || c.now < 0 || c.old > cap || c.now > cap ? (int64_t)1 << 40 : grow;
    x[1] += max(c.held - c.want, 0);
    x[2] += b < upto ? grow : 0;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
    if (lane == 0) words[k][warp] = x[k];
  }
  __syncthreads();
  Totals t{0, 0, 0, false};
  for (int i = 0; i < kThr / 32; ++i) {
    t.grow += words[0][i];
    t.less += words[1][i];
    t.grow_before += words[2][i];
  }
  // pages given back must not reach those handed out
  t.ok = first >= 0 && first < a.n_free && count >= 0 && t.grow <= count && count + t.less <= a.n_free;
  return t;
}

// entry i of the ring, i below 3 n
__device__ __forceinline__ int32_t* ring(const AssignArgs& a, int64_t i) {
  i -= i >= a.n_free ? a.n_free : 0;
  return a.free_pages + (i >= a.n_free ? i - a.n_free : i);
}
// Token t of sequence b: its place, and its slot; the sequence's first new page is the ring's entry `from`.
__device__ __forceinline__ void place(const AssignArgs& a, const Change& c, int b, int t, int64_t from, bool ok) {
  const int64_t at = (int64_t)b * a.T + t;
  int64_t slot = -1;
  int pos = -1;
  if (ok && t < c.now - c.old) {
    pos = c.old + t;
    const int j = whole_pages(a, pos);
    const int page = j < c.held ? a.table[(int64_t)b * a.table_stride + j] : *ring(a, from + (j - c.held));
    slot = (int64_t)page * a.page_size + (pos - j * a.page_size);
  }
  a.slots[at] = slot;
  a.positions[at] = pos;
}

// Block x places the tokens from x % chunks * kPlaceTokens on of `per` sequences (one, unless there are thousands).
__device__ __forceinline__ void place_tokens(const AssignArgs& a, int x, int chunks, int per, int64_t (*words)[kThreads / 32]) {
  const int b0 = x / chunks * per, t0 = x % chunks * kPlaceTokens;
  const int first = a.state[0], count = a.state[1];
  const Totals all = totals_of<kThreads>(a, first, count, b0, words);
  const int end = min(a.T, t0 + kPlaceTokens);
  int64_t from = (int64_t)first + all.grow_before;
  for (int b = b0; b < min(a.B, b0 + per); ++b) {
    const Change c = change_of(a, b);
#pragma unroll 4
    for (int t = t0 + threadIdx.x; t < end; t += kThreads) place(a, c, b, t, from, all.ok);
    from += max(c.want - c.held, 0);
  }
}

// Block 0 (of all launches' blocks, from `begin` on): tables, ring, lengths and state, and where `places` the tokens too.
// The others place tokens.
__global__ void __launch_bounds__(kThreads) assign_kernel(const AssignArgs a, const int begin, const bool places, const int chunks,
                                                          const int per) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int64_t words[3][kWarps];
  if (begin + (int)blockIdx.x > 0) {
    place_tokens(a, begin + (int)blockIdx.x - 1, chunks, per, words);
    return;
  }
  __shared__ int scan[2][kWarps];
  __shared__ Change changes[kThreads];
  __shared__ int grown[kThreads], given[kThreads];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int first = a.state[0], count = a.state[1];
  const Totals all = totals_of<kThreads>(a, first, count, 0, words);
  const bool ok = all.ok;
  if (!ok && threadIdx.x == 0) atomicExch(a.err, kDevBadOffsets);

  int G = 0, R = 0;                                        // of the sequences before the chunk
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x, nb = min(kThreads, a.B - b0);
    Change c{0, 0, 0, 0};
    if (b < a.B && ok) c = change_of(a, b);
    int up = max(c.want - c.held, 0), down = max(c.held - c.want, 0);
    const int up0 = up, down0 = down;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, up, o), y = __shfl_up_sync(0xffffffffu, down, o);
      if (lane >= o) {
        up += x;
        down += y;
      }
    }
    if (b0 > 0) __syncthreads();                           // the chunk before is done with
    if (lane == 31) {
      scan[0][warp] = up;
      scan[1][warp] = down;
    }
    __syncthreads();
    int base_up = G, base_down = R;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        base_up += scan[0][w];
        base_down += scan[1][w];
      }
      G += scan[0][w];
      R += scan[1][w];
    }
    const int before = base_up + up - up0, behind = base_down + down - down0;
    changes[threadIdx.x] = c;
    grown[threadIdx.x] = before;
    given[threadIdx.x] = behind;
    if (b < a.B) a.q_lens[b] = ok ? max(c.now - c.old, 0) : 0;
    // a page or two more, or less: the sequence's own thread
    const bool few = abs(c.want - c.held) <= 2;
    if (few) {
      int32_t* const row = a.table + (int64_t)b * a.table_stride;
      for (int j = c.held; j < c.want; ++j) row[j] = *ring(a, (int64_t)first + before + (j - c.held));
      for (int j = c.want; j < c.held; ++j) *ring(a, (int64_t)first + count + behind + (j - c.want)) = row[j];
    }
    // many: a warp takes the sequence
    __syncthreads();
    if (ok)
      for (int i = warp; i < nb; i += kWarps) {
        const Change d = changes[i];
        if (abs(d.want - d.held) <= 2) continue;
        int32_t* const row = a.table + (int64_t)(b0 + i) * a.table_stride;
        for (int j = d.held + lane; j < d.want; j += 32) row[j] = *ring(a, (int64_t)first + grown[i] + (j - d.held));
        for (int j = d.want + lane; j < d.held; j += 32) *ring(a, (int64_t)first + count + given[i] + (j - d.want)) = row[j];
      }
    if (places)
      for (int x = threadIdx.x; x < nb * a.T; x += kThreads) {
        const int i = a.T == 1 ? x : x / a.T;
        place(a, changes[i], b0 + i, x - i * a.T, (int64_t)first + grown[i], ok);
      }
  }
  // lengths and state may be written over those that were read
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    const int n = ok ? a.new_lens[b] : a.old_lens[b];
    a.lens[b] = n;
  }
  if (threadIdx.x == 0) {
    const int64_t f = (int64_t)first + (ok ? all.grow : 0);
    a.state_out[0] = (int)(ok && f >= a.n_free ? f - a.n_free : f);
    a.state_out[1] = ok ? (int)(count - all.grow + all.less) : count;
  }
}

}  // namespace

cudaError_t launch_assign(const AssignArgs& args, cudaStream_t s) {
  AssignArgs a = args;
  a.page_magic = ((uint64_t(1) << 43) + a.page_size - 1) / a.page_size;
  if ((int64_t)a.B * a.T <= 4 * kThreads) {                // one block places them too
    assign_kernel<<<1, kThreads, 0, s>>>(a, 0, true, 1, 1);
    return cudaGetLastError();
  }
  const int chunks = (a.T + kPlaceTokens - 1) / kPlaceTokens;
  const int per = (a.B + 4095) / 4096, groups = (a.B + per - 1) / per;     // (each block reads all lengths)
  const int64_t blocks = (int64_t)groups * chunks;
  if (blocks >= 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (a.lens != a.old_lens && a.lens != a.new_lens && a.state_out != a.state) {
    assign_kernel<<<(unsigned)blocks + 1, kThreads, 0, s>>>(a, 0, false, chunks, per);
    return cudaGetLastError();
  }
  assign_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(a, 1, false, chunks, per);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  assign_kernel<<<1, kThreads, 0, s>>>(a, 0, false, chunks, per);
  return cudaGetLastError();
}

}  // namespace fa
