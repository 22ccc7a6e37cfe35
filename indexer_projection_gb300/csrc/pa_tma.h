// Host-side TMA tensor maps shared by the kernels that load tiles with
// cp.async.bulk.tensor: the driver's encoder (looked up once through the
// runtime, so the library needs no link against libcuda) and the two map
// shapes the kernels use.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace pa {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// [rows, row_bytes] bytes, row-major: boxes of box_rows rows x box_bytes
// (<= 128) bytes, 128-byte swizzle (16-byte chunk c of row r lands at chunk
// c ^ (r % 8) of its 128-byte line), rows past the end read as zero.
inline bool map_rows_sw128(CUtensorMap *map, const void *base, uint64_t rows, uint64_t row_bytes, uint32_t box_bytes,
                           uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {box_bytes, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// F8_128x4 scale atoms as a [row blocks, ksf*16] int64 grid: one box = one
// 512-byte atom (128 rows x 4 K-blocks); row blocks past the end read as zero.
inline bool map_scale_atoms(CUtensorMap *map, const void *base, int row_blocks, int ksf) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)ksf * 16, (cuuint64_t)row_blocks};
  cuuint64_t strides[1] = {(cuuint64_t)ksf * 128};
  cuuint32_t box[2] = {64, 1};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of row_bytes (a multiple of 16) in pages: dim 0 a row, dim 1 the
// page's rows (row_bytes apart), dim 2 the pages (page_bytes apart); one box
// is box_rows rows of each of box_pages pages, in that order.
inline bool map_page_rows(CUtensorMap *map, const void *base, uint32_t row_bytes, uint64_t rows, uint64_t page_bytes,
                          uint64_t pages, uint32_t box_rows, uint32_t box_pages) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)row_bytes / 8, (cuuint64_t)rows, (cuuint64_t)pages};
  cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)page_bytes};
  cuuint32_t box[3] = {row_bytes / 8, box_rows, box_pages};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_INT64, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pa
