// tensor_maps.cuh -- host side: tensor maps of byte matrices in boxes 128 bytes wide with the
// 128-byte swizzle, zeros outside; and the shared-memory limit of kernels.  The driver's encoder is looked up at run time, so the library
// does not link against the driver.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static std::atomic<void*> entry{nullptr};
    void* p = entry.load(std::memory_order_relaxed);
    if (!p) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess)
            return nullptr;
        entry.store(p, std::memory_order_relaxed);
    }
    return (EncodeTiled)p;
}

inline bool make_map(CUtensorMap* map, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box) {
    const EncodeTiled enc = encode_tiled();
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(p), dims, strides, box,
                      unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows][bytes] in boxes of box_rows rows
inline bool make_rows_map(CUtensorMap* map, const void* p, int64_t rows, int64_t bytes, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    return make_map(map, p, 2, dims, strides, box);
}

// [E][rows][bytes] in boxes of box_rows rows of one expert
inline bool make_experts_map(CUtensorMap* map, const void* p, int64_t E, int64_t rows, int64_t bytes, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)bytes, (cuuint64_t)rows, (cuuint64_t)E};
    const cuuint64_t strides[2] = {(cuuint64_t)bytes, (cuuint64_t)(rows * bytes)};
    const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
    return make_map(map, p, 3, dims, strides, box);
}

// [E][gate, up][n][bytes] in boxes of `pairs` gates and then their ups
inline bool make_pairs_map(CUtensorMap* map, const void* p, int64_t E, int64_t n, int64_t bytes, int pairs) {
    const cuuint64_t dims[4] = {(cuuint64_t)bytes, (cuuint64_t)n, 2, (cuuint64_t)E};
    const cuuint64_t strides[3] = {(cuuint64_t)bytes, (cuuint64_t)(n * bytes), (cuuint64_t)(2 * n * bytes)};
    const cuuint32_t box[4] = {128, (cuuint32_t)pairs, 2, 1};
    return make_map(map, p, 4, dims, strides, box);
}

// Allows `kernel` `bytes` of dynamic shared memory: the first time on each device, which `done`
// (one of the kernel's own) remembers.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit & done.load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace
