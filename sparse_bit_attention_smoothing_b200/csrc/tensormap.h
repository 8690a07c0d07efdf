// tensormap.h -- tensor maps (TMA descriptors) on the host.  The driver's
// encoder is found through the runtime, so the library needs no libcuda at
// link time.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

namespace sagesla {

// A map of `rank` dimensions, the innermost contiguous; `strides` in bytes of
// the others, elements outside read as zeros.  False: refused by the driver.
inline bool tensor_map(CUtensorMap* m, const void* p, CUtensorMapDataType type, int rank, const unsigned long* dims,
                       const unsigned long* strides, const unsigned* box, CUtensorMapSwizzle swizzle) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  cuuint64_t d[5], s[5];
  cuuint32_t b[5], one[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    one[i] = 1;
    if (i + 1 < rank) s[i] = strides[i];
  }
  return encode(m, type, (cuuint32_t)rank, const_cast<void*>(p), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sagesla
