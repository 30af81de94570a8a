// Attention over a cache of int8 pages, whole or chosen ones (fa_paged_kernel.cuh).
#include "fa_paged_kernel.cuh"

namespace fa {

cudaError_t launch_paged_int8(const PagedArgs& a, cudaStream_t s) { return paged8<FA_PAGES_INT8>(a, s); }

}  // namespace fa
