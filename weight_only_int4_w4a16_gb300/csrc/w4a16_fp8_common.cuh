// Shared by the 8-bit linear's two kernels: 16-bit conversions, status bits and
// the tensor maps of their operands.
#pragma once

#include "w4a16_internal.h"

namespace w4a16 {

// device status bits: a wait for a stage, for a block's sums, for a free stage
// expired; something in flight did not land before the exit
constexpr int kErrStageWait = 1 << 17, kErrSumWait = 1 << 18, kErrSlotWait = 1 << 19,
              kErrDrain = 1 << 20;

__device__ __forceinline__ float half_bits_to_float(uint16_t h, int bf16) {
    return bf16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}
__device__ __forceinline__ uint16_t float_to_half_bits(float v, int bf16) {  // nearest even
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
                : __half_as_ushort(__float2half_rn(v));
}

// 8-bit rows [rows, K] in boxes of box_rows rows x 128 k, 128-byte swizzle; what a
// box has past the end comes as zeros
inline bool encode_fp8_rows(CUtensorMap *map, const void *base, int rows, int K, int box_rows) {
    const EncodeTiledFn encode = tensor_map_encoder();
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {(cuuint32_t)kGroup, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims,
                            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 16-bit rows [rows, cols] (cols a multiple of 8, base 16-byte aligned) in boxes of
// box_rows x box_cols, 128-byte swizzle; what a box has past the end is not stored
// (and comes as zeros)
inline bool encode_rows16(CUtensorMap *map, const void *base, int rows, int cols, int box_rows,
                          int box_cols) {
    const EncodeTiledFn encode = tensor_map_encoder();
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims,
                            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_NONE,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace w4a16
