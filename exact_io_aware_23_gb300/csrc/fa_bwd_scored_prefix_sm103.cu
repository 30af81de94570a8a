// The two-pass backward's kernels (fa_bwd_split_sm103.cuh) with a prefix alone.
#include "fa_bwd_split_sm103.cuh"

namespace fa {

cudaError_t launch_bwd_scored_prefix(const BwdArgs& a, const BwdMaps& m, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_FP16)
    return a.d == 64 ? launch_bwd_split<64, true, false, kModPrefix>(a, m, s) : launch_bwd_split<128, true, false, kModPrefix>(a, m, s);
  return a.d == 64 ? launch_bwd_split<64, false, false, kModPrefix>(a, m, s) : launch_bwd_split<128, false, false, kModPrefix>(a, m, s);
}

}  // namespace fa
