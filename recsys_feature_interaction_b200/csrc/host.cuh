// host.cuh -- the host-side helpers that the library's source files share: the per-device
// context, shared-memory limits, tensor maps and launch status. Defined in wk_api.cu.
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"
#include "wukong.h"

namespace wk {

struct DevInfo {
  bool init = false;
  int id = 0;
  int sms = 0;
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  unsigned* standalone_status = nullptr;  // the status word of the stand-alone calls
};

// The current device's context (set up on the first call).
wk_status dev_info(DevInfo** out);

// Raises the dynamic shared-memory limit of a kernel once per device.
wk_status smem_attr(const DevInfo* dv, const void* fn, int bytes);

// Tiled tensor map; dims[0] is the contiguous dimension, strides in bytes for dims 1..rank-1.
bool make_map(const DevInfo* dv, CUtensorMap* m, CUtensorMapDataType dt, uint32_t rank, const void* base,
              const uint64_t* dims, const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle sw);

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline wk_status launch_status() {
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? WK_OK : WK_ERR_CUDA;
}

template <typename T>
constexpr CUtensorMapDataType tmap_dtype() {
  return sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                        : (Half16<T>::kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
}
template <>
constexpr CUtensorMapDataType tmap_dtype<float>() {
  return CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
}

}  // namespace wk
