// tensor_maps.h -- TMA descriptors of the GEMMs' operands, scale tiles and outputs (host side).
#pragma once

#include "bsp_internal.h"

namespace bsp {

enum Kind : int { kNVF4 = 0, kMXF8 = 1 };

// Row-major uint8 matrix [rows, row_bytes], boxes of box_rows x box_bytes (128
// or 64) with the matching TMA swizzle.
inline int encode_operand(CUtensorMap* m, const void* base, int64_t rows, int64_t row_bytes, int box_rows,
                          int box_bytes = 128) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1u, 1u};
  CUresult r = encode_tiled_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE,
                                 box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSP_OK : BSP_ERR_INVALID_ARG;
}

// Row-major bytes [rows, row_bytes], boxes of box_rows x box_bytes, no swizzle.
inline int encode_rows_plain(CUtensorMap* m, const void* base, int64_t rows, int64_t row_bytes, int box_rows, int box_bytes) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1u, 1u};
  CUresult r = encode_tiled_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSP_OK : BSP_ERR_INVALID_ARG;
}

// Tile-mapped scale buffer viewed as [bands][tiles per band][512 bytes] with
// 8-byte elements; a box covers `atoms` consecutive 512-byte tiles of `bands`
// consecutive row bands.
inline int encode_scales(CUtensorMap* m, const void* base, int64_t bands, int64_t tiles_per_band, int atoms, int box_bands) {
  cuuint64_t dims[3] = {64u, static_cast<cuuint64_t>(tiles_per_band), static_cast<cuuint64_t>(bands)};
  cuuint64_t strides[2] = {512u, static_cast<cuuint64_t>(tiles_per_band * 512)};
  cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(atoms), static_cast<cuuint32_t>(box_bands)};
  cuuint32_t es[3] = {1u, 1u, 1u};
  CUresult r = encode_tiled_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<void*>(base), dims, strides, box, es,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSP_OK : BSP_ERR_INVALID_ARG;
}

// Row-major output [rows, ld] of bf16 or fp32, boxes of box_rows rows x box_cols columns (32, 64 or 128 bytes, with
// the swizzle of that width).
inline int encode_rows(CUtensorMap* m, void* base, int64_t rows, int64_t cols, int64_t ld, bool f32, int box_rows,
                       int box_cols) {
  const int64_t esize = f32 ? 4 : 2;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * esize)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1u, 1u};
  const int64_t bytes = box_cols * esize;
  const CUtensorMapSwizzle swizzle = bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_32B;
  CUresult r = encode_tiled_fn()(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base,
                                 dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                                 CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSP_OK : BSP_ERR_INVALID_ARG;
}

// Weights stacked by expert, [experts][rows, row_bytes] without gaps: boxes of box_rows rows x 128 bytes of one
// expert, 128-byte swizzle.  Rows past an expert's last read as zeros, not as the next expert's.
inline int encode_experts(CUtensorMap* m, const void* base, int64_t experts, int64_t rows, int64_t row_bytes,
                          int box_rows) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(experts)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows * row_bytes)};
  cuuint32_t box[3] = {128u, static_cast<cuuint32_t>(box_rows), 1u};
  cuuint32_t es[3] = {1u, 1u, 1u};
  CUresult r = encode_tiled_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSP_OK : BSP_ERR_INVALID_ARG;
}

// The same weights with rows alternating between a gate and an up projection, boxes of 128 rows taken as 8 blocks of
// 8 gate rows and 8 up rows (rows % 16 == 0).
inline int encode_experts_gated(CUtensorMap* m, const void* base, int64_t experts, int64_t rows, int64_t row_bytes) {
  cuuint64_t dims[5] = {static_cast<cuuint64_t>(row_bytes), 8u, 2u, static_cast<cuuint64_t>(rows / 16),
                        static_cast<cuuint64_t>(experts)};
  cuuint64_t strides[4] = {static_cast<cuuint64_t>(2 * row_bytes), static_cast<cuuint64_t>(row_bytes),
                           static_cast<cuuint64_t>(16 * row_bytes), static_cast<cuuint64_t>(rows * row_bytes)};
  cuuint32_t box[5] = {128u, 8u, 2u, 8u, 1u};
  cuuint32_t es[5] = {1u, 1u, 1u, 1u, 1u};
  CUresult r = encode_tiled_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(base), dims, strides, box, es,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSP_OK : BSP_ERR_INVALID_ARG;
}

// Their scale buffers, [experts][bands][tiles per band][512 bytes]: boxes of `atoms` tiles of one band.
inline int encode_expert_scales(CUtensorMap* m, const void* base, int64_t experts, int64_t bands,
                                int64_t tiles_per_band, int atoms) {
  cuuint64_t dims[4] = {64u, static_cast<cuuint64_t>(tiles_per_band), static_cast<cuuint64_t>(bands),
                        static_cast<cuuint64_t>(experts)};
  cuuint64_t strides[3] = {512u, static_cast<cuuint64_t>(tiles_per_band * 512),
                           static_cast<cuuint64_t>(bands * tiles_per_band * 512)};
  cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(atoms), 1u, 1u};
  cuuint32_t es[4] = {1u, 1u, 1u, 1u};
  CUresult r = encode_tiled_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 4, const_cast<void*>(base), dims, strides, box, es,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSP_OK : BSP_ERR_INVALID_ARG;
}

}  // namespace bsp
