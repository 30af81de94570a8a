// Attention over chosen pages of a 16-bit cache (fa_paged_kernel.cuh).
#include "fa_paged_kernel.cuh"

namespace fa {

cudaError_t launch_paged_picked(const PagedArgs& a, fa_dtype dt, cudaStream_t s) {
  if (dt == FA_FP16)
    return a.d == 64 ? paged<Cfg<64, FA_PAGES_16BIT, true, true>>(a, s) : paged<Cfg<128, FA_PAGES_16BIT, true, true>>(a, s);
  return a.d == 64 ? paged<Cfg<64, FA_PAGES_16BIT, false, true>>(a, s) : paged<Cfg<128, FA_PAGES_16BIT, false, true>>(a, s);
}

}  // namespace fa
