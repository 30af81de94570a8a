// Attention over a cache of e4m3 pages, whole or chosen ones (fa_paged_kernel.cuh).
#include "fa_paged_kernel.cuh"

namespace fa {

cudaError_t launch_paged_e4m3(const PagedArgs& a, cudaStream_t s) { return paged8<FA_PAGES_E4M3>(a, s); }

}  // namespace fa
