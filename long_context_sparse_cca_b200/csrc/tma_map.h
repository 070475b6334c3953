// Host helper: TMA tensor maps over [planes, rows, d] tensors of 16-bit
// elements (bf16 or fp16), as the tcgen05 kernels read them: 64 x 128 x 1
// boxes (one 128-byte row of 64 elements per box line), 128-byte swizzle,
// zero fill outside the tensor.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime_api.h>

#include <cstdint>

namespace cca {

inline PFN_cuTensorMapEncodeTiled_v12000 tma_encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    return fn;
}

// row_stride, plane_stride: in elements, multiples of 8; 0: contiguous.
inline bool make_map(CUtensorMap *m, const void *ptr, int d, int64_t rows, int64_t planes,
                     bool f16 = false, int64_t row_stride = 0, int64_t plane_stride = 0)
{
    auto fn = tma_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                          static_cast<cuuint64_t>(planes)};
    cuuint64_t strides[2] = {
        static_cast<cuuint64_t>(row_stride ? row_stride : d) * 2,
        static_cast<cuuint64_t>(plane_stride ? plane_stride : static_cast<int64_t>(rows) * d) * 2};
    cuuint32_t box[3] = {64, 128, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          3, const_cast<void *>(ptr), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

}  // namespace cca
