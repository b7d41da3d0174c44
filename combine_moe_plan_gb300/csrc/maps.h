// maps.h -- host side of the TMA kernels: tensor maps, and the device's SMs.
#pragma once

#include <cstddef>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime (no driver library is linked);
// NULL if there is none.  Looked up once.
inline EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// A map of a dense [rows, width] tensor of bytes, bf16 or fp32, in boxes of box_rows x
// 128 bytes, 128-byte swizzle; a load reads zeros past the end.
inline bool tile_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, size_t rows, int width, int box_rows) {
    const EncodeTiledFn encode = encode_tiled();
    if (encode == nullptr) return false;
    const int size = type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 1 : type == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 2 : 4;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width * size};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows}, steps[2] = {1, 1};
    return encode(m, type, 2, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of a dense [rows, width] bf16 tensor whose rows are a product's inner
// dimension: boxes of box_rows by 128 elements, stored as two blocks of 64
// elements (128 bytes, 128-byte swizzle) by box_rows.  The coordinates are
// (0, row, element / 64); a load reads zeros past either end.
inline bool block_map(CUtensorMap* m, const void* base, size_t rows, int width, int box_rows) {
    const EncodeTiledFn encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)width / 64}, strides[2] = {(cuuint64_t)width * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 2}, steps[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same over a window of rows that ends anywhere: the coordinates are (0, i, row,
// element / 64) with `window` values of i, and row + i is the row in memory.  A box
// (window rows) that begins at i = -z has z rows of zeros, then window - z rows from
// `row` on, and touches no row behind them.
inline bool window_map(CUtensorMap* m, const void* base, size_t rows, int width, int window) {
    const EncodeTiledFn encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t pitch = (cuuint64_t)width * 2;
    const cuuint64_t dims[4] = {64, (cuuint64_t)window, (cuuint64_t)rows, (cuuint64_t)width / 64}, strides[3] = {pitch, pitch, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)window, 1, 2}, steps[4] = {1, 1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device (0: none).
inline int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return sms;
}

}  // namespace moe
