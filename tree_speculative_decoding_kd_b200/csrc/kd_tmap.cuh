// Tensor maps (host) for the kernels' TMA boxes of bf16 rows, 128-byte swizzle.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kd_common.cuh"

namespace kd {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// bf16 view [n2][n1][inner] with strides s1, s2 in elements (multiples of 8); boxes of
// 64 x b1 x b2 elements.  A stride of an axis of length 1 (or 0) is never used, so it may be anything.
inline int make_tmap3(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t n1, uint64_t n2, int64_t s1, int64_t s2,
                      uint32_t b1, uint32_t b2) {
  auto fn = tmap_encode_fn();
  if (!fn) {
    set_cuda_error(cudaErrorNotSupported, "cuTensorMapEncodeTiled");
    return KD_ELAUNCH;
  }
  const cuuint64_t dims[3] = {inner, n1 ? n1 : 1, n2 ? n2 : 1};
  const cuuint64_t strides[2] = {(cuuint64_t)(n1 > 1 ? s1 * 2 : (int64_t)inner * 2),
                                 (cuuint64_t)(n2 > 1 ? s2 * 2 : (int64_t)inner * 2)};
  const cuuint32_t box[3] = {64, b1, b2}, es[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
    return KD_ELAUNCH;
  }
  return KD_OK;
}

}  // namespace kd
