// Attention over a cache of int8 pages, whole or chosen ones (fa_paged_kernel.cuh).
#include "fa_paged_kernel.cuh"

namespace fa {

cudaError_t launch_paged_int8(const PagedArgs& a, cudaStream_t s) {
  if (a.pages != nullptr)
    return a.d == 64 ? paged<Cfg<64, FA_PAGES_INT8, true, true>>(a, s) : paged<Cfg<128, FA_PAGES_INT8, true, true>>(a, s);
  return a.d == 64 ? paged<Cfg<64, FA_PAGES_INT8, true, false>>(a, s) : paged<Cfg<128, FA_PAGES_INT8, true, false>>(a, s);
}

}  // namespace fa
