// Host helpers shared by the TMA kernels' launchers (defined in gmm_tc.cu).
#pragma once

#include <cudaTypedefs.h>

namespace moe {
namespace tc {

// cuTensorMapEncodeTiled, looked up once; nullptr if the driver lacks it.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
// MOE_OK on an sm_103 device, else MOE_ERR_UNSUPPORTED or MOE_ERR_CUDA.
int device_ok();

// Dense tensor map; dims innermost first, in elements of `esz` bytes (1: bytes,
// 2: bf16).
inline bool make_map(CUtensorMap* m, const void* ptr, int esz, int rank, const uint64_t* dims,
                     const uint32_t* box, CUtensorMapSwizzle swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t gdim[3], gstride[2];
  cuuint32_t bdim[3], estr[3] = {1, 1, 1};
  uint64_t stride = (uint64_t)esz;
  for (int i = 0; i < rank; ++i) {
    gdim[i] = dims[i];
    bdim[i] = box[i];
    if (i > 0) gstride[i - 1] = stride;
    stride *= dims[i];
  }
  return fn(m, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
            const_cast<void*>(ptr), gdim, gstride, bdim, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// With 128-byte swizzle.
inline bool make_map_sw128(CUtensorMap* m, const void* ptr, int esz, int rank, const uint64_t* dims,
                           const uint32_t* box) {
  return make_map(m, ptr, esz, rank, dims, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace tc
}  // namespace moe
