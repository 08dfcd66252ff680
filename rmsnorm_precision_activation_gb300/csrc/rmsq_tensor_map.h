// rmsq_tensor_map.h -- tensor maps for TMA loads of row-major codes and scales.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace rmsq {

// cuTensorMapEncodeTiled from the driver (the library does not link it).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn()
{
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load();
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f);
    }
    return reinterpret_cast<EncodeFn>(f);
}

// A matrix [rows x columns] of elements of 1 or 8 bytes, read in boxes of box_rows x box_columns; what lies outside
// reads as 0.
inline bool encode_map(CUtensorMap* map, const void* data, int element_bytes, long long rows, long long columns, int box_rows,
                       int box_columns, CUtensorMapSwizzle swizzle)
{
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(columns) * static_cast<cuuint64_t>(element_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_columns), static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
    const auto make = [&]() {
        return fn(map, element_bytes == 8 ? CU_TENSOR_MAP_DATA_TYPE_UINT64 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                  const_cast<void*>(data), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    const CUresult r = make();
    if (r != CUDA_ERROR_INVALID_CONTEXT) return r == CUDA_SUCCESS;
    // a thread that has made no runtime call that binds the device's context yet
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && make() == CUDA_SUCCESS;
}

}  // namespace rmsq
