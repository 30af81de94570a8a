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
// bytes of the slots.  One cluster of blocks; each sums up all lengths for itself, and only what may be the
// caller's own input (lengths, ring state) is written behind a barrier of the cluster.
#include <cuda_runtime.h>

#include "fa_paged.cuh"
#include "fa_sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;                // of a cluster

__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Change {
  int old, now, held, want;
};
__device__ __forceinline__ Change change_of(const AssignArgs& a, int b) {
  Change c;
  c.old = a.old_lens[b];
  c.now = a.new_lens[b];
  // sums in 64 bits: lengths reach to 2^31 - 1
  c.held = (int)(((int64_t)c.old + a.page_size - 1) / a.page_size);
  c.want = (int)(((int64_t)c.now + a.page_size - 1) / a.page_size);
  return c;
}

// The block's sum of x.
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* words) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if (lane == 0) words[warp] = x;
  __syncthreads();
  int64_t sum = 0;
  for (int i = 0; i < kWarps; ++i) sum += words[i];
  return sum;
}

__global__ void __launch_bounds__(kThreads) assign_kernel(const AssignArgs a) {
  __shared__ int64_t words[kWarps];
  __shared__ int scan[2][kWarps];
  __shared__ int olds[kThreads], news[kThreads], grown[kThreads], given[kThreads];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x, ctas = (int)cluster_ctas();
  const int first = a.state[0], count = a.state[1];
  const int64_t cap = (int64_t)a.max_pages * a.page_size;

  // whether all of it can be done
  int64_t grow = 0, less = 0, bad = 0;
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    const Change c = change_of(a, b);
    bad += c.old < 0 || c.now < 0 || c.old > cap || c.now > cap;
    grow += max(c.want - c.held, 0);
    less += max(c.held - c.want, 0);
  }
  grow = block_sum(grow, words);
  less = block_sum(less, words);
  bad = block_sum(bad, words);
  const bool ok = bad == 0 && first >= 0 && first < a.n_free && count >= 0 && grow <= count && count - grow + less <= a.n_free &&
                  count + less <= a.n_free;
  if (!ok && cta == 0 && threadIdx.x == 0) atomicExch(a.err, kDevBadOffsets);
  const int64_t all = (int64_t)cta * kThreads + threadIdx.x, threads = (int64_t)ctas * kThreads;
  auto ring = [&](int64_t i) {                             // i below 3 n
    i -= i >= a.n_free ? a.n_free : 0;
    return a.free_pages + (i >= a.n_free ? i - a.n_free : i);
  };

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
    __syncthreads();                                       // the chunk before is done with
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
    olds[threadIdx.x] = c.old;
    news[threadIdx.x] = c.now;
    grown[threadIdx.x] = base_up + up - up0;
    given[threadIdx.x] = base_down + down - down0;
    __syncthreads();

    // pages: a warp takes a sequence
    if (ok)
      for (int i = cta * kWarps + warp; i < nb; i += ctas * kWarps) {
        int32_t* const row = a.table + (int64_t)(b0 + i) * a.table_stride;
        const int held = (int)(((int64_t)olds[i] + a.page_size - 1) / a.page_size);
        const int want = (int)(((int64_t)news[i] + a.page_size - 1) / a.page_size);
        for (int j = held + lane; j < want; j += 32) row[j] = *ring((int64_t)first + grown[i] + (j - held));
        for (int j = want + lane; j < held; j += 32) *ring((int64_t)first + count + given[i] + (j - want)) = row[j];
      }
    // places of the new tokens
    const int64_t tokens = (int64_t)nb * a.T;
    for (int64_t x = all; x < tokens; x += threads) {
      const int i = (int)(x / a.T), t = (int)(x - (int64_t)i * a.T);
      const int64_t at = (int64_t)(b0 + i) * a.T + t;
      const int pos = olds[i] + t;
      int64_t slot = -1;
      if (ok && t < news[i] - olds[i]) {
        const int held = (int)(((int64_t)olds[i] + a.page_size - 1) / a.page_size), j = pos / a.page_size;
        const int page = j < held ? a.table[(int64_t)(b0 + i) * a.table_stride + j]
                                  : *ring((int64_t)first + grown[i] + (j - held));
        slot = (int64_t)page * a.page_size + (pos - j * a.page_size);
      }
      a.slots[at] = slot;
      a.positions[at] = slot < 0 ? -1 : pos;
    }
    for (int64_t i = all; i < nb; i += threads) a.q_lens[b0 + i] = ok ? max(news[i] - olds[i], 0) : 0;
  }
  // lengths and state may be written over those that were read
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  for (int64_t b = all; b < a.B; b += threads) {
    const int n = ok ? a.new_lens[b] : a.old_lens[b];
    a.lens[b] = n;
  }
  if (all == 0) {
    int64_t f = (int64_t)first + (ok ? grow : 0);
    a.state_out[0] = (int)(ok && f >= a.n_free ? f - a.n_free : f);
    a.state_out[1] = ok ? (int)(count - grow + less) : count;
  }
}

}  // namespace

cudaError_t launch_assign(const AssignArgs& a, cudaStream_t s) {
  // a block for every 2048 tokens' places
  const int64_t work = (int64_t)a.B * a.T;
  int ctas = 1;
  while (ctas < kMaxCtas && ctas * (int64_t)2048 < work) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, assign_kernel, a);
}

}  // namespace fa
