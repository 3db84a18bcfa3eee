// Tensor maps of the uncompressed key/value kernels (host side).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "internal.h"

namespace tpla {

// Stride in bytes of a dimension with `n` entries of 16-bit elements; one
// entry is never stepped over, and its stride may be anything.
inline cuuint64_t map_stride(int64_t n, int64_t stride) {
  return n > 1 ? (cuuint64_t)stride * 2 : 16;
}

inline bool encode_16bit_5d(CUtensorMap* map, const void* base, bool f16, const cuuint64_t (&dims)[5],
                            const cuuint64_t (&strides)[4], const cuuint32_t (&box)[5]) {
  PFN_cuTensorMapEncodeTiled_v12000 enc =
      reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
  return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
             const_cast<void*>(base), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Keys or values [pages, rows, heads, D] (one "page" for packed rows) as
// (column, row, 64-column chunk, head, page); a box is 64 rows of
// `box_chunks` chunks of one head.  An empty tensor is never read: its map
// stands on `placeholder`, with one entry in each empty dimension.
inline bool encode_kv_tiles(CUtensorMap* map, const void* base, const void* placeholder, bool f16,
                            int64_t rows, int64_t heads, int64_t pages, int64_t s0, int64_t s1,
                            int64_t s2, int D, int box_chunks) {
  const bool none = rows == 0 || pages == 0;
  const cuuint64_t dims[5] = {64, (cuuint64_t)(rows > 0 ? rows : 1), (cuuint64_t)(D / 64),
                              (cuuint64_t)heads, (cuuint64_t)(pages > 0 ? pages : 1)};
  const cuuint64_t strides[4] = {map_stride(rows, s1), 128, map_stride(heads, s2),
                                 map_stride(pages, s0)};
  const cuuint32_t box[5] = {64, 64, (cuuint32_t)box_chunks, 1, 1};
  return encode_16bit_5d(map, none ? placeholder : base, f16, dims, strides, box);
}

}  // namespace tpla
