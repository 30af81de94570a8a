// The two-pass backward's kernels (fa_bwd_split_sm103.cuh) with scores capped by a tanh.
#include "fa_bwd_split_sm103.cuh"

namespace fa {

cudaError_t launch_bwd_scored_cap(const BwdArgs& a, const BwdMaps& m, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_FP16)
    return a.d == 64 ? launch_bwd_split<64, true, false, kModCap>(a, m, s) : launch_bwd_split<128, true, false, kModCap>(a, m, s);
  return a.d == 64 ? launch_bwd_split<64, false, false, kModCap>(a, m, s) : launch_bwd_split<128, false, false, kModCap>(a, m, s);
}

}  // namespace fa
