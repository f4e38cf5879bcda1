// attn_tc.cuh -- what the tcgen05 attention kernels over 16-bit caches share: a tile of 128 rows by 128 keys of
// head_dim 128, its products and its softmax (tree_attn_tc.cu describes the roles).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "sm100.cuh"

namespace eagle {
namespace attn_tc {

using namespace sm100;

constexpr int KT = 128;                   // keys per tile
constexpr int HALF = 16384;               // one 64-dim half of a 128-row tile (bytes)
constexpr int TILE = 2 * HALF;            // one K or V tile
constexpr float kRescaleLog2 = 8.f;       // lazy rescale threshold (log2 units)

// Bits 0..n-1 set (n clamped to [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Scores of keys whose bit is clear become -inf.
__device__ __forceinline__ void mask_keys(uint32_t (&r)[32], uint32_t bits) {
#pragma unroll
  for (int j = 0; j < 32; ++j) r[j] = ((bits >> j) & 1u) ? r[j] : 0xff800000u;
}

// Maximum of 64 floats with three-input max instructions, as a shallow tree.
__device__ __forceinline__ float max64(const uint32_t (&a)[32], const uint32_t (&b)[32]) {
  float m[22];
#pragma unroll
  for (int i = 0; i < 10; ++i)
    m[i] = max3(__uint_as_float(a[3 * i]), __uint_as_float(a[3 * i + 1]), __uint_as_float(a[3 * i + 2]));
  m[10] = max3(__uint_as_float(a[30]), __uint_as_float(a[31]), __uint_as_float(b[0]));
#pragma unroll
  for (int i = 0; i < 10; ++i)
    m[11 + i] = max3(__uint_as_float(b[3 * i + 1]), __uint_as_float(b[3 * i + 2]), __uint_as_float(b[3 * i + 3]));
  m[21] = fmaxf(__uint_as_float(b[31]), m[0]);
  float n[7];
#pragma unroll
  for (int i = 0; i < 7; ++i) n[i] = max3(m[3 * i + 1], m[3 * i + 2], m[3 * i + 3]);
  return max3(max3(n[0], n[1], n[2]), max3(n[3], n[4], n[5]), n[6]);
}

// S (TMEM columns scol) = Q K^T over the 8 K-steps of 16 head dims.
__device__ __forceinline__ void issue_qk(uint32_t tb, const uint8_t* sQ, const uint8_t* sK, uint32_t scol) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, KT, 0, 0);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint32_t off = (ks >> 2) * HALF + (ks & 3) * 32;
    mma_ss(tb + scol, smem_desc_sw128(smem_u32(sQ) + off, 16, 1024), smem_desc_sw128(smem_u32(sK) + off, 16, 1024),
           idesc, ks > 0);
  }
}

// O (TMEM columns ocol) += P V over the 8 K-steps of 16 keys; the P of keys
// 64 h + 16 k .. sits in columns scol + 64 h + 8 k .. (the precise low parts 32 columns
// further on).
template <bool PRECISE>
__device__ __forceinline__ void issue_pv(uint32_t tb, const uint8_t* sV, uint32_t scol, uint32_t ocol, bool first) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 1);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint64_t bd = smem_desc_sw128(smem_u32(sV) + ks * 2048, HALF, 1024);
    const uint32_t acol = scol + (ks >> 2) * 64 + (ks & 3) * 8;
    mma_ts(tb + ocol, tb + acol, bd, idesc, (first && ks == 0) ? 0u : 1u);
    if constexpr (PRECISE) mma_ts(tb + ocol, tb + acol + 32, bd, idesc, 1u);
  }
}

// P of 32 keys held in registers (raw scores, masked keys -inf) -> TMEM columns
// `col` .. (bf16 pairs; the precise low parts 32 columns further on), 16 keys per
// store.  Returns the fp32 row sum of the 32 values.
template <bool PRECISE>
__device__ __forceinline__ float emit_p32(const uint32_t (&r)[32], uint32_t col, uint64_t sl2x2, uint64_t nmux2) {
  float sum = 0.f;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t hi[8], lo[8];
    uint64_t acc2 = 0ull;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = 16 * g + 2 * j;
      float x0, x1;
      f32x2_split(fma_f32x2(f32x2(r[k], r[k + 1]), sl2x2, nmux2), x0, x1);
      const float p0 = ex2(x0), p1 = ex2(x1);
      __nv_bfloat162 u = __floats2bfloat162_rn(p0, p1);
      hi[j] = *reinterpret_cast<uint32_t*>(&u);
      if constexpr (PRECISE) {
        const float h0 = __uint_as_float(hi[j] << 16), h1 = __uint_as_float(hi[j] & 0xffff0000u);
        __nv_bfloat162 w = __floats2bfloat162_rn(p0 - h0, p1 - h1);
        lo[j] = *reinterpret_cast<uint32_t*>(&w);
      }
      // the row sum adds the fp32 p: hi + lo differs from p by at most 2^-17 p
      acc2 = add_f32x2(acc2, f32x2(__float_as_uint(p0), __float_as_uint(p1)));
    }
    tmem_st8(col + 8 * g, hi);
    if constexpr (PRECISE) tmem_st8(col + 32 + 8 * g, lo);
    float a0, a1;
    f32x2_split(acc2, a0, a1);
    sum += a0 + a1;
  }
  return sum;
}

}  // namespace attn_tc
}  // namespace eagle
