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

// Rows of `dim` (64 or 128) bf16 elements as [dim / 64][rows][64], boxes of all halves of `box_rows` rows, each
// half's rows of 128 bytes swizzled; zero fill.
inline bool make_tmap_halves(CUtensorMap* m, const void* base, int dim, unsigned long long rows, unsigned box_rows) {
  auto fn = tmap_encode_fn();
  if (!fn) return false;
  const unsigned halves = static_cast<unsigned>(dim) / 64;
  const cuuint64_t dims[3] = {64, rows, halves};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(dim) * 2, 128};
  const cuuint32_t box[3] = {64, box_rows, halves};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace eagle
