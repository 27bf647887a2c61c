// Tensor maps of bf16 tiles: what every tensor copy of this library reads through.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace mla {

// A map of a bf16 tensor (dims and box innermost first, strides in bytes from the second dimension on) whose boxes land
// 128-byte swizzled; elements past the end read as zeros.  False if the driver lacks the encoder or refuses the map.
inline bool encode_bf16_map(CUtensorMap *m, const void *ptr, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                            const cuuint32_t *box) {
    // Looked up once; the initialisation of a function-local static is thread-safe.
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
    return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(ptr), dims, strides, box,
                            steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mla
