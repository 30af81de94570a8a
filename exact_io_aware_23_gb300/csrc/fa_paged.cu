// Attention over a paged cache: the kernel for 16-bit pages, and the host's side of all of them.
#include <atomic>
#include <chrono>

#include "fa_paged_kernel.cuh"

namespace fa {

int paged_ctas() {
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess || sms <= 0) sms = 152;      // GB300's when no device can be asked
  return sms * kCtasPerSm;
}

unsigned long long paged_call_number() {
  static std::atomic<unsigned long long> next{
      (unsigned long long)std::chrono::system_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15ull};
  const unsigned long long n = next.fetch_add(1, std::memory_order_relaxed);
  return n != 0 ? n : paged_call_number();             // 0 is a cleared word
}

// Whether CTAs share segments.  Few segments of at most 512 keys get a CTA each, at most two after one
// another in an SM's places: nothing to reckon, nothing to join and no workspace.
bool paged_shares(int B, int Hkv, int rows, int capacity, int ctas) {
  const int64_t segments = (int64_t)B * Hkv * ((rows + kRows - 1) / kRows);
  return capacity > 512 || segments > 2 * (int64_t)ctas;
}

// Whether the units of all segments can be counted in 31 bits.
bool paged_counts(int B, int Hkv, int rows, int capacity, bool bits8) {
  const int64_t segments = (int64_t)B * Hkv * ((rows + kRows - 1) / kRows);
  return segments <= 0x7fffffff / ((int64_t)capacity / 16 + 1 + (bits8 ? kFlipSegment : kSegment));
}

// The workspace: arrivals [2 * ctas], then two parts of 16 rows a CTA, their statistics and outputs.
// Variants with more and smaller CTAs have as many rows of parts, and their arrivals fit too.
PagedWorkspace paged_workspace(int ctas, int d) {
  PagedWorkspace w;
  const size_t rows = 2 * (size_t)ctas * kRows;
  static_assert(flip_ctas(64) * 8 <= kCtasPerSm * kRows && flip_ctas(128) * 8 <= kCtasPerSm * kRows, "parts of 8 rows take the place of those of 16");
  w.ml = (2 * (size_t)ctas * 2 * sizeof(unsigned long long) + 255) / 256 * 256;
  w.o = w.ml + rows * sizeof(float2);
  w.total = (w.o + rows * d * sizeof(float) + 255) / 256 * 256;
  return w;
}

cudaError_t launch_paged(const PagedArgs& a, fa_dtype dt, cudaStream_t s) {
  if (a.store == FA_PAGES_E4M3) return launch_paged_e4m3(a, s);
  if (a.store == FA_PAGES_INT8) return launch_paged_int8(a, s);
  if (a.pages != nullptr) return launch_paged_picked(a, dt, s);
  if (dt == FA_FP16)
    return a.d == 64 ? paged<Cfg<64, FA_PAGES_16BIT, true, false>>(a, s) : paged<Cfg<128, FA_PAGES_16BIT, true, false>>(a, s);
  return a.d == 64 ? paged<Cfg<64, FA_PAGES_16BIT, false, false>>(a, s) : paged<Cfg<128, FA_PAGES_16BIT, false, false>>(a, s);
}

}  // namespace fa
