// The two-pass backward's kernels (fa_bwd_split_sm103.cuh) with a bias linear in distance.
#include "fa_bwd_split_sm103.cuh"

namespace fa {

cudaError_t launch_bwd_scored_bias(const BwdArgs& a, const BwdMaps& m, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_FP16)
    return a.d == 64 ? launch_bwd_split<64, true, false, kModBias>(a, m, s) : launch_bwd_split<128, true, false, kModBias>(a, m, s);
  return a.d == 64 ? launch_bwd_split<64, false, false, kModBias>(a, m, s) : launch_bwd_split<128, false, false, kModBias>(a, m, s);
}

}  // namespace fa
