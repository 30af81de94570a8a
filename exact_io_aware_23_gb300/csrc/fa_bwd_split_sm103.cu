// The two-pass backward's kernels without score modifications (fa_bwd_split_sm103.cuh), and the
// choice among all of them.
#include "fa_bwd_split_sm103.cuh"

namespace fa {

cudaError_t launch_bwd_split_sm103(const BwdArgs& a, fa_dtype dt, cudaStream_t s) {
  if (a.scored) {
    // no tile mask or dropout with score modifications
    if (a.drop.enabled || a.block_mask != nullptr) return cudaErrorInvalidValue;
    switch (mod_of(a.score)) {
      case kModCap: return launch_bwd_scored_cap(a, dt, s);
      case kModBias: return launch_bwd_scored_bias(a, dt, s);
      case kModBoth: return launch_bwd_scored_both(a, dt, s);
      default: return launch_bwd_scored_prefix(a, dt, s);
    }
  }
  if (a.drop.enabled) {
    if (dt == FA_FP16)
      return a.d == 64 ? launch_bwd_split<64, true, true, kModNone>(a, s) : launch_bwd_split<128, true, true, kModNone>(a, s);
    return a.d == 64 ? launch_bwd_split<64, false, true, kModNone>(a, s) : launch_bwd_split<128, false, true, kModNone>(a, s);
  }
  if (dt == FA_FP16)
    return a.d == 64 ? launch_bwd_split<64, true, false, kModNone>(a, s) : launch_bwd_split<128, true, false, kModNone>(a, s);
  return a.d == 64 ? launch_bwd_split<64, false, false, kModNone>(a, s) : launch_bwd_split<128, false, false, kModNone>(a, s);
}

}  // namespace fa
