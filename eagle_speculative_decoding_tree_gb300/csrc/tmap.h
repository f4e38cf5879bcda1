// tmap.h -- tensor maps of the 8-bit and the paged KV cache kernels (host).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace eagle {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// [rows][cols] row-major elements of `esz` bytes, boxes of box_cols x box_rows, zero fill.
inline bool make_tmap_2d(CUtensorMap* m, CUtensorMapDataType dt, int esz, const void* base, unsigned long long cols,
                         unsigned long long rows, unsigned box_cols, unsigned box_rows, CUtensorMapSwizzle sw) {
  auto fn = tmap_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * static_cast<unsigned>(esz)};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t es[2] = {1, 1};
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of `dim` (64 or 128) bf16 (esz 2) or fp32 (4) elements in parts of 128 bytes, [parts][rows][128 bytes]; boxes of
// all parts of `box_rows` rows, each part's rows swizzled; zero fill.
inline bool make_tmap_halves(CUtensorMap* m, const void* base, int dim, unsigned long long rows, unsigned box_rows,
                             int esz = 2) {
  auto fn = tmap_encode_fn();
  if (!fn) return false;
  const unsigned per = 128u / esz, parts = static_cast<unsigned>(dim) / per;
  const cuuint64_t dims[3] = {per, rows, parts};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(dim) * esz, 128};
  const cuuint32_t box[3] = {per, box_rows, parts};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base),
            dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace eagle
