// The two-pass backward's kernels without score modifications (fa_bwd_split_sm103.cuh), and the
// choice among all of them.
#include "fa_bwd_split_sm103.cuh"

namespace fa {
namespace {

cudaError_t make_map(CUtensorMap* m, const void* base, int D, int N, int BH, bool f16) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)BH};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)N * D * 2};
  const cuuint32_t box[3] = {64, 128, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_tensor_map(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           3, base, dims, strides, box, estr, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t make_bwd_maps(const BwdArgs& a, fa_dtype dt, BwdMaps* m) {
  // token axis and slice count of the tensor maps: per (b, h) slice, or packed per head
  const bool packed = a.cu_seqlens != nullptr, f16 = dt == FA_FP16;
  const int q_slices = packed ? a.H : a.B * a.H, kv_slices = packed ? a.Hkv : a.B * a.Hkv;
  cudaError_t e;
  if ((e = make_map(&m->q, a.q, a.d, a.rows, q_slices, f16)) != cudaSuccess) return e;
  if ((e = make_map(&m->k, a.k, a.d, a.rows, kv_slices, f16)) != cudaSuccess) return e;
  if ((e = make_map(&m->v, a.v, a.d, a.rows, kv_slices, f16)) != cudaSuccess) return e;
  return make_map(&m->dO, a.dO, a.d, a.rows, q_slices, f16);
}

cudaError_t launch_bwd_split_sm103(const BwdArgs& a, const BwdMaps& m, fa_dtype dt, cudaStream_t s) {
  if (a.scored) {
    // no tile mask or dropout with score modifications
    if (a.drop.enabled || a.block_mask != nullptr) return cudaErrorInvalidValue;
    switch (mod_of(a.score)) {
      case kModCap: return launch_bwd_scored_cap(a, m, dt, s);
      case kModBias: return launch_bwd_scored_bias(a, m, dt, s);
      case kModBoth: return launch_bwd_scored_both(a, m, dt, s);
      default: return launch_bwd_scored_prefix(a, m, dt, s);
    }
  }
  if (a.drop.enabled) {
    if (dt == FA_FP16)
      return a.d == 64 ? launch_bwd_split<64, true, true, kModNone>(a, m, s) : launch_bwd_split<128, true, true, kModNone>(a, m, s);
    return a.d == 64 ? launch_bwd_split<64, false, true, kModNone>(a, m, s) : launch_bwd_split<128, false, true, kModNone>(a, m, s);
  }
  if (dt == FA_FP16)
    return a.d == 64 ? launch_bwd_split<64, true, false, kModNone>(a, m, s) : launch_bwd_split<128, true, false, kModNone>(a, m, s);
  return a.d == 64 ? launch_bwd_split<64, false, false, kModNone>(a, m, s) : launch_bwd_split<128, false, false, kModNone>(a, m, s);
}

}  // namespace fa
