// Which of several blocks comes last: a word of a workspace counts those that have written their part,
// {the call's number, the count}, whatever a fresh workspace holds.
//
// Each block sees to the number early (by one compare-and-swap from whatever the word holds, unless another
// block was first), so that its end takes one fence and one addition.  The number has 48 bits, starts at
// another place in every process and is not used twice in one (paged_call_number); the block that comes last
// clears the word, for a captured call's next run under the same number.  Nobody waits.
#pragma once

#include <cuda_runtime.h>

namespace fa {
namespace {

__device__ __forceinline__ void open_count(unsigned long long* word, unsigned long long call) {
  unsigned long long w;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(word) : "memory");
  if ((w ^ (call << 16)) >> 16 != 0) atomicCAS(word, w, call << 16);
}
// True for the last of `parts` (below 2^16).  What the block wrote is released before, and the others' parts acquired
// behind, by the caller's fences.
__device__ __forceinline__ bool count_part(unsigned long long* word, int parts) {
  return (int)(atomicAdd(word, 1ull) & 0xffffu) == parts - 1;
}

}  // namespace
}  // namespace fa
