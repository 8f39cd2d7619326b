// tensor_map.h -- the driver's encoder of TMA tensor maps, for the operators of
// sequence models (found through the runtime: no link-time dependency on libcuda).
// Not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace fftgb {

using TensorMapEncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                       const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                       const cuuint32_t *, CUtensorMapInterleave,
                                       CUtensorMapSwizzle, CUtensorMapL2promotion,
                                       CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, or null.
inline TensorMapEncodeFn tensor_map_encode() {
  static TensorMapEncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<TensorMapEncodeFn>(nullptr);
    return reinterpret_cast<TensorMapEncodeFn>(p);
  }();
  return fn;
}

}  // namespace fftgb
