// Host-side construction of TMA tensor maps for the operators around the scan.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "train_ops.h"

namespace ttm {

bool make_tma_map(void* map, TmaType type, const void* ptr, const unsigned long long (&dims)[3],
                  const unsigned long long (&strides)[2], const unsigned (&box)[3], bool swizzle128) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!encode) return false;
    const CUtensorMapDataType t = type == TmaType::f32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : type == TmaType::bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t d[3] = {dims[0], dims[1], dims[2]}, s[2] = {strides[0], strides[1]};
    const cuuint32_t b[3] = {box[0], box[1], box[2]}, e[3] = {1, 1, 1};
    return encode(static_cast<CUtensorMap*>(map), t, 3, const_cast<void*>(ptr), d, s, b, e,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ttm
