// Host side of the TMA tensor copies: 2-D tiled tensor maps over row-major
// bf16 matrices in this GPU's memory, encoded through the driver entry point
// that the runtime hands out (no link against the driver library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

namespace dbc {
namespace tma {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline void *driver_entry(const char *name) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint(name, &p, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess
               ? p : nullptr;
}

// The encoder, or NULL.  It is a driver call and needs a context on the calling host thread, which a
// thread whose first CUDA call this is does not have yet: the runtime's device is then made current (legal
// in a stream capture; a context that is there already stays).
inline EncodeFn encoder() {
    using CurrentFn = CUresult (*)(CUcontext *);
    static EncodeFn fn = nullptr;
    static CurrentFn current = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        fn = reinterpret_cast<EncodeFn>(driver_entry("cuTensorMapEncodeTiled"));
        current = reinterpret_cast<CurrentFn>(driver_entry("cuCtxGetCurrent"));
    });
    CUcontext ctx = nullptr;
    int dev = 0;
    if (current && (current(&ctx) != CUDA_SUCCESS || !ctx) &&
        (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess)) {
        cudaGetLastError();                              // not the next call's
        return nullptr;
    }
    return fn;
}

// Tensor map of a row-major bf16 matrix [rows][cols] (cols * 2 bytes a
// multiple of 16, base 16-byte aligned) read in boxes of box_rows x 64
// columns with the 128-byte swizzle: one box lands as box_rows rows of 128
// bytes, the 16-byte chunk c of row r at chunk c ^ (r % 8).  Out-of-range rows
// read as zeros.  Returns false when the encoder is unavailable or refuses.
inline bool encode_bf16_rows(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of a row-major fp32 matrix [rows][cols] (cols * 4 bytes a multiple of 16, base 16-byte
// aligned) in boxes of box_rows x 32 columns (128 bytes) with the 128-byte swizzle, for tile
// stores from shared memory.
inline bool encode_f32_rows(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * 4};
    const cuuint32_t box[2] = {32, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of row-major 8-bit rows of K bytes, `ld` bytes apart (a multiple of 16, base 16-byte
// aligned), read in boxes of box_rows x 128 bytes with the 128-byte swizzle.  Bytes past K and rows
// past the end read as zeros.
inline bool encode_i8_rows(CUtensorMap *map, const void *base, uint64_t rows, uint64_t K, uint64_t ld,
                           uint32_t box_rows) {
    EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {K, rows};
    const cuuint64_t strides[1] = {ld};
    const cuuint32_t box[2] = {128, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of row-major fp32 or bf16 rows of `cols` elements, `ld` elements apart (row starts on
// 16-byte boundaries), for tile stores of box_rows x 64 bytes with the 64-byte swizzle (chunk c of row
// r at c ^ (r / 2 % 4)).
inline bool encode_out_rows(CUtensorMap *map, void *base, bool bf16, uint64_t rows, uint64_t cols, uint64_t ld,
                            uint32_t box_rows) {
    EncodeFn fn = encoder();
    if (!fn) return false;
    const uint32_t esz = bf16 ? 2 : 4;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {ld * esz};
    const cuuint32_t box[2] = {64 / esz, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tma
}  // namespace dbc
