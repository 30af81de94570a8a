// The deterministic backward's two tensor-core passes in one launch: the key-stationary dK/dV
// pass (fa_dkdv_sm103.cuh) and the query-stationary dQ pass (fa_dq_sm103.cuh).
//
// The passes are independent once D = rowsum(dO * O) exists, read the same four tensors and
// need one SM each (a CTA of either kind holds most of the shared memory and all of TMEM).  In
// one grid, the dK/dV CTAs come first and the dQ CTAs after them, so the last wave of the first
// pass is filled with the second pass's CTAs instead of idling.  (Alternating the two kinds
// CTA by CTA was measured 30 % slower: each kind then streams its slice's tiles at half the
// rate, and the tiles no longer stay in L2 between the CTAs that share them.)
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_dkdv_sm103.cuh"
#include "fa_dq_sm103.cuh"
#include "fa_internal.cuh"
#include "fa_sm103.cuh"

namespace fa {
namespace {

// Both passes run with BwdLayout<D>'s block, one CTA per SM: at d = 128 320 threads (10 warps,
// three on some of the SM's four 16K-register partitions, so at most 16384 / 96 -> 168
// registers a thread), at d = 64 576 (18 warps, at most 112).
template <int D, bool F16, bool kDrop, int kMod>
__global__ void __launch_bounds__(BwdLayout<D>::kThreads, 1)
bwd_split_sm103_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                       const BwdArgs a, const int n_kv_units, const int n_q_units) {
  (void)n_q_units;
  // under a tile mask, a plan may reorder the units so that the longest start first
  const int x = a.perm != nullptr ? a.perm[blockIdx.x] : (int)blockIdx.x;
  if (x < n_kv_units) dkdv::run<D, F16, kDrop, kMod>(x, tmQ, tmK, tmV, tmDO, a);
  else dqp::run<D, F16, kDrop, kMod>(x - n_kv_units, tmQ, tmK, tmV, tmDO, a);
}

template <int D, bool F16, bool kDrop, int kMod>
cudaError_t launch_bwd_split(const BwdArgs& a, const BwdMaps& m, cudaStream_t s) {
  const int BH = a.B * a.H;            // query-side work units per tile row (Q, dO, dQ)
  const int BHkv = a.B * a.Hkv;        // key/value-side work units per tile row (K, V, dK, dV)
  cudaError_t e;
  auto kern = bwd_split_sm103_kernel<D, F16, kDrop, kMod>;
  // each pass keeps its barriers 256 bytes below its live-tile bitmap (one bit per tile)
  const int bitmap = a.block_mask != nullptr ? ((a.n_tiles + 127) / 128) * 16 : 0;
  int smem = max(dkdv::Cfg<D, F16>::kSmem, dqp::Cfg<D, F16>::kSmem);
  smem = max(smem, dkdv::Cfg<D, F16>::kBar + 256 + bitmap);
  smem = max(smem, dqp::Cfg<D, F16>::kBar + 256 + bitmap);
  static LaunchSetup setup;
  if ((e = prepare_launch(setup, kern, smem)) != cudaSuccess) return e;
  const int n_t = (a.N + 127) / 128;
  const int n_kv = n_t * BHkv, n_q = n_t * BH;
  kern<<<dim3(n_kv + n_q), BwdLayout<D>::kThreads, smem, s>>>(m.q, m.k, m.v, m.dO, a, n_kv, n_q);
  return cudaGetLastError();
}

}  // namespace
}  // namespace fa
