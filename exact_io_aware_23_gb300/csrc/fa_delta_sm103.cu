// D = rowsum(P * dP) for the scored backward, on the tensor cores (bf16 or fp16 in, fp32
// accumulate), d in {64, 128}.
//
// The softmax's gradient is dS = P (dP - D) with D_i = sum_j P_ij dP_ij, which equals dO_i . O_i.
// Taken from the stored O it inherits that tensor's rounding and that of the probabilities O was
// summed from: D is then off by a few 2^-9 of |dO . O|, the same error for all of a row's keys, and
// where few keys carry a row (a steep distance bias, short rows, peaked scores) this outweighs all
// other roundings of dQ and dK: it made their error 1.5 to 2.2 times that of fp32 arithmetic
// rounded at the end, 1.4 without it.  So D is summed here from P and dP themselves, in fp32, as
// they come out of the tensor cores: two products more than the backward's seven, no pass over O.
//
// One CTA = two 128-row query tiles of one (b, h) slice, 384 threads:
//   warp 8      TMA producer: Q_0, Q_1, dO_0, dO_1 once, then K_j, V_j in turn through one ring
//   warp 9      MMA issuer (one thread): S_t = Q_t K_j^T, then dP_t = dO_t V_j^T, t = 0, 1
//   warps 0-3   query tile 0, warps 4-7 query tile 1; a thread owns a row (a TMEM lane): 128 scores
//               to registers, which frees S_t for the next key tile at once, P, then dP 32 columns
//               at a time into the row's sum.
//   warps 10, 11 only make up the third warpgroup, which gives registers to the other two.
//   TMEM (512 columns): S_0, S_1, dP_0, dP_1, 128 each.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include "fa_internal.cuh"
#include "fa_score.cuh"
#include "fa_sm103.cuh"
#include "ptx_sm103.cuh"

namespace fa {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

enum : int { kNone = 0, kPartial = 1, kFull = 2 };

template <int D, bool F16>
struct Cfg {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kSlots = D == 128 ? 3 : 8;            // K and V tiles in turn
  static constexpr int kQ = 0;                               // Q_t at kQ + t * kTile
  static constexpr int kDO = 2 * kTile;                      // dO_t at kDO + t * kTile
  static constexpr int kRing = 4 * kTile;
  static constexpr int kBar = kRing + kSlots * kTile;
  static constexpr int kSmem = kBar + 256;
  static constexpr uint32_t kS = 0, kDP = 256;               // TMEM columns of tile t: + 128 t
  static constexpr uint32_t kIdesc = ptx::idesc_f32acc(128, 128, false, false, F16);
};

struct Bars {
  uint64_t q_full;
  uint64_t full[8];        // ring
  uint64_t empty[8];
  uint64_t s_full[2], s_free[2];
  uint64_t dp_full[2], dp_free[2];
  uint64_t done;
  uint64_t tail;           // the last V tile, before its rows behind the keys are cleared
  uint32_t tmem_base;
};
static_assert(sizeof(Bars) <= 256, "");

template <int D, bool F16, int kMod>
__global__ void __launch_bounds__(kThreads, 1)
delta_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO, const BwdArgs a) {
  using C = Cfg<D, F16>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {      // the operand tiles need 1 KB alignment
    if (threadIdx.x == 0) atomicExch(a.err, kDevMisaligned);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBar);
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t lim_ms = a.dbg.wait_limit_ms;
  // Work order as the forward's: under a mask slices vary fastest and the longest pairs go first.
  const int BH = a.B * a.H, n_pairs = (a.N + 2 * BM - 1) / (2 * BM);
  const int bh = a.heads_fastest ? blockIdx.x % BH : blockIdx.x / n_pairs;
  const int at = a.heads_fastest ? blockIdx.x / BH : blockIdx.x % n_pairs;
  const int q0 = (a.causal ? n_pairs - 1 - at : at) * 2 * BM;
  const int b = bh / a.H, h = bh % a.H;
  int row0 = 0, N = a.N;
  if (a.cu_seqlens != nullptr) {
    if (!packed_sequence(a.cu_seqlens, b, a.N, a.rows, &row0, &N)) {
      if (threadIdx.x == 0) atomicExch(a.err, kDevBadOffsets);
      return;
    }
    if (q0 >= N) return;
  }
  const int qs = a.cu_seqlens != nullptr ? h : bh;
  const int ks = (a.cu_seqlens != nullptr ? 0 : b * a.Hkv) + h / (a.H / a.Hkv);
  int kv_lim = N;
  if (a.kv_lens != nullptr) kv_lim = max(0, min(a.N, (int)a.kv_lens[b]));
  const int prefix = a.causal && a.score.prefix != nullptr ? min(max(a.score.prefix[b], 0), N) : 0;
  int last = kv_lim;
  if (a.causal) last = min(last, max(min(q0 + 2 * BM, N), prefix));
  const int tiles = (last + BN - 1) / BN;
  const bool has_tail = tiles * BN > kv_lim && (a.cu_seqlens != nullptr ? row0 + kv_lim < a.rows : kv_lim < a.N);

  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_u32(&bars->q_full), 1);
    for (int s = 0; s < C::kSlots; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bars->s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->s_free[t]), 4);
      ptx::mbar_init(ptx::smem_u32(&bars->dp_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->dp_free[t]), 4);
    }
    ptx::mbar_init(ptx::smem_u32(&bars->done), 1);
    ptx::mbar_init(ptx::smem_u32(&bars->tail), 1);
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp >= 8) {
    ptx::regs_dec<88>();
  if (warp == 8) {
    // ------------------------------- TMA producer -----------------------------------------------
    int m = 0;                                     // tiles issued: K_0, V_0, K_1, ...
    if (lane == 0 && tiles > 0) {
      const uint32_t qb = ptx::smem_u32(&bars->q_full);
      ptx::mbar_arrive_expect_tx(qb, 4 * C::kTile);
      for (int t = 0; t < 2; ++t)
        for (int hh = 0; hh < D / 64; ++hh) {
          ptx::tma_load_3d(sbase + C::kQ + t * C::kTile + hh * 128 * 128, &tmQ, qb, hh * 64, row0 + q0 + t * BM, qs);
          ptx::tma_load_3d(sbase + C::kDO + t * C::kTile + hh * 128 * 128, &tmDO, qb, hh * 64, row0 + q0 + t * BM, qs);
        }
      for (; m < 2 * tiles; ++m) {
        const int slot = m % C::kSlots;
        if (!ptx::mbar_wait(ptx::smem_u32(&bars->empty[slot]), ((uint32_t)(m / C::kSlots) & 1u) ^ 1u, lim_ms, a.err)) break;
        const uint32_t fb = ptx::smem_u32(has_tail && m == 2 * tiles - 1 ? &bars->tail : &bars->full[slot]);
        ptx::mbar_arrive_expect_tx(fb, C::kTile);
        for (int hh = 0; hh < D / 64; ++hh)
          ptx::tma_load_3d(sbase + C::kRing + slot * C::kTile + hh * 128 * 128, (m & 1) ? &tmV : &tmK, fb, hh * 64,
                           row0 + (m >> 1) * BN, ks);
      }
    }
    if (has_tail && __shfl_sync(0xffffffffu, m, 0) == 2 * tiles) {
      // the values behind the keys meet probabilities of 0, and 0 * NaN is not 0: cleared first
      const int slot = (2 * tiles - 1) % C::kSlots;
      ptx::mbar_wait(ptx::smem_u32(&bars->tail), 0, lim_ms, a.err);
      zero_rows<D>(smem + C::kRing + slot * C::kTile, kv_lim - (tiles - 1) * BN);
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->full[slot]));
    }
    if (lane == 0 && tiles > 0) {
      // drain: copies in flight must land before shared memory is released
      ptx::mbar_wait(ptx::smem_u32(&bars->q_full), 0, lim_ms, a.err);
      for (int i = max(0, m - C::kSlots); i < m; ++i)
        ptx::mbar_wait(ptx::smem_u32(&bars->full[i % C::kSlots]), (uint32_t)(i / C::kSlots) & 1u, lim_ms, a.err);
    }
  } else if (warp == 9) {
    // ------------------------------- MMA issuer -------------------------------------------------
    if (lane == 0) {
      bool ok = tiles == 0 || ptx::mbar_wait(ptx::smem_u32(&bars->q_full), 0, lim_ms, a.err);
      // n-th pair of products of one kind: dst_t = A_t (ring tile m)^T, each after the warps have
      // read the last one's result
      auto products = [&](int n, int m, uint32_t dst, uint32_t src, uint64_t* full, uint64_t* free) -> bool {
        const int slot = m % C::kSlots;
        if (!ptx::mbar_wait(ptx::smem_u32(&bars->full[slot]), (uint32_t)(m / C::kSlots) & 1u, lim_ms, a.err)) return false;
        const uint32_t sb = sbase + C::kRing + slot * C::kTile;
        for (int t = 0; t < 2; ++t) {
          if (n > 0 && !ptx::mbar_wait(ptx::smem_u32(&free[t]), (uint32_t)(n - 1) & 1u, lim_ms, a.err)) return false;
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * (128 * 128) + (kk % 4) * 32;
            ptx::mma_ss(tmem + dst + t * 128, ptx::sdesc_sw128(sbase + src + t * C::kTile + off, 16, 1024),
                        ptx::sdesc_sw128(sb + off, 16, 1024), C::kIdesc, kk > 0);
          }
          ptx::mma_commit(ptx::smem_u32(&full[t]));
        }
        return true;
      };
      for (int n = 0; n < tiles && ok; ++n) {
        ok = products(n, 2 * n, C::kS, C::kQ, bars->s_full, bars->s_free);
        if (ok) ok = products(n, 2 * n + 1, C::kDP, C::kDO, bars->dp_full, bars->dp_free);
      }
      ptx::mma_commit(ptx::smem_u32(&bars->done));
      ptx::mbar_wait(ptx::smem_u32(&bars->done), 0, lim_ms, a.err);
    }
  }
  } else {
    ptx::regs_inc<200>();
    // ------------------------------- rows -------------------------------------------------------
    const int t = warp / 4, sub = warp % 4;
    const int i = q0 + t * BM + sub * 32 + lane;
    const uint32_t lane_off = (uint32_t)(sub * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::kS + t * 128, tP = tmem + lane_off + C::kDP + t * 128;
    const float c = a.scale * kLog2e;
    const float m = (kMod & kModCap) == 0 ? c : a.score.cap_log2;
    const float2 m2 = make_float2(m, m);
    const size_t row = (size_t)qs * a.rows + row0 + i;
    const float L = i < N ? a.lse[row] : -INFINITY;
    const float nl = L == -INFINITY ? -INFINITY : -L * kLog2e;     // P vanishes on empty rows
    const float2 nl2 = make_float2(nl, nl);
    const float slope = (kMod & kModBias) != 0 ? a.score.slopes[h] * kLog2e : 0.f;
    const int seen = a.causal ? min(kv_lim, max(i + 1, prefix)) : kv_lim;        // keys of the row
    const int r0 = q0 + t * BM, r1 = min(r0 + BM, N) - 1;
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    for (int n = 0; n < tiles; ++n) {
      const int c0 = n * BN, c1 = c0 + BN - 1;
      int kind = kPartial;
      if (r0 >= N || (a.causal && c0 > r1 && c0 >= prefix)) kind = kNone;
      else if (c1 < kv_lim && (!a.causal || c1 <= r0 || c1 < prefix)) kind = kFull;
      if (!ptx::mbar_wait(ptx::smem_u32(&bars->s_full[t]), (uint32_t)n & 1u, lim_ms, a.err)) break;
      ptx::tc_fence_after();
      float p[BN];
      if (kind != kNone) {
        uint32_t raw[4][32];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) ptx::tmem_ld32(tS + q4 * 32, raw[q4]);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          ptx::reg_fence(raw[q4]);
#pragma unroll
          for (int e = 0; e < 32; ++e) p[q4 * 32 + e] = __uint_as_float(raw[q4][e]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(ptx::smem_u32(&bars->s_free[t]));
        // S_1(n) has completed, and S_0(n) before it: K_n's slot is free
        if (t == 1 && sub == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->empty[(2 * n) % C::kSlots]));
      }
      if (kind != kNone) {
        // what is masked, or no row, does not choose the form of the tanh for the others
        const int lim = i < N ? seen - c0 : 0;
        if (kind == kPartial || r1 - r0 < BM - 1) {
#pragma unroll
          for (int e = 0; e < BN; ++e) p[e] = e < lim ? p[e] : 0.f;
        }
        const int lo = c0 - (r0 + BM - 1), hi = lo + BM + BN - 2;              // of j - i in the tile
        const Bias bi = make_bias(slope, c0 - i, lo, a.causal && prefix == 0 ? min(hi, 0) : hi);
        with_score<kMod>(p, a.score, F16 ? a.score.poly_limit : a.score.low_limit, bi, [&](auto cap, auto bias) {
          constexpr int kCap = decltype(cap)::value, kBias = decltype(bias)::value;
#pragma unroll
          for (int col = 0; col < BN; col += 2) {
            float2 x = make_float2(p[col], p[col + 1]);
            if constexpr (kCap != kCapNone) x = tanh_of<kCap, F16>(x, a.score);
            x = ptx::fma2(x, m2, nl2);
            if constexpr (kBias != kBiasNone) x = biased<kBias>(x, bi, col);
            p[col] = ptx::ex2(x.x);
            p[col + 1] = ptx::ex2(x.y);
          }
        });
        if (kind == kPartial) {
#pragma unroll
          for (int e = 0; e < BN; ++e) p[e] = e < lim ? p[e] : 0.f;
        }
      }
      if (!ptx::mbar_wait(ptx::smem_u32(&bars->dp_full[t]), (uint32_t)n & 1u, lim_ms, a.err)) break;
      ptx::tc_fence_after();
      if (kind != kNone) {
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t raw[32];
          ptx::tmem_ld32(tP + q4 * 32, raw);
          ptx::tmem_wait_ld();
          ptx::reg_fence(raw);
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            sum[(e >> 1) & 1] = ptx::fma2(make_float2(p[q4 * 32 + e], p[q4 * 32 + e + 1]),
                                          make_float2(__uint_as_float(raw[e]), __uint_as_float(raw[e + 1])), sum[(e >> 1) & 1]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(ptx::smem_u32(&bars->dp_free[t]));
        // dP_1(n) has completed, and dP_0(n) before it: V_n's slot is free
        if (t == 1 && sub == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->empty[(2 * n + 1) % C::kSlots]));
      }
    }
    if (i < N) a.delta[row] = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 9) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool F16, int kMod>
cudaError_t launch(const BwdArgs& a, const BwdMaps& m, cudaStream_t s) {
  cudaError_t e;
  auto kern = delta_kernel<D, F16, kMod>;
  static LaunchSetup setup;
  // The warp groups re-split the CTA's registers; that only completes if the launch holds them.
  int regs = 0;
  if ((e = prepare_launch(setup, kern, Cfg<D, F16>::kSmem, &regs)) != cudaSuccess) return e;
  if (regs * kThreads < 128 * 88 + 256 * 200) return cudaErrorInvalidConfiguration;
  kern<<<dim3((a.N + 2 * BM - 1) / (2 * BM) * a.B * a.H), kThreads, Cfg<D, F16>::kSmem, s>>>(m.q, m.k, m.v, m.dO, a);
  return cudaGetLastError();
}

template <int kMod>
cudaError_t dispatch(const BwdArgs& a, const BwdMaps& m, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_FP16) return a.d == 64 ? launch<64, true, kMod>(a, m, s) : launch<128, true, kMod>(a, m, s);
  return a.d == 64 ? launch<64, false, kMod>(a, m, s) : launch<128, false, kMod>(a, m, s);
}

}  // namespace

cudaError_t launch_delta_sm103(const BwdArgs& a, const BwdMaps& m, fa_dtype dt, cudaStream_t s) {
  switch (mod_of(a.score)) {
    case kModCap: return dispatch<kModCap>(a, m, dt, s);
    case kModBias: return dispatch<kModBias>(a, m, dt, s);
    case kModBoth: return dispatch<kModBoth>(a, m, dt, s);
    default: return dispatch<kModPrefix>(a, m, dt, s);
  }
}

}  // namespace fa
