// paged.cuh -- device helpers of the paged KV cache kernels.
#pragma once

#include "common.cuh"
#include "paged.h"
#include "sm100.cuh"

namespace eagle {

// Row number in the pool ([n_pages][Hkv][T] rows) of cache row r, KV head h, of request b, -1 if its
// page is not in the pool.  0 <= r < capacity.
__device__ __forceinline__ int paged_row(const PagedGeom& g, int b, int h, int r) {
  const int page = g.table[static_cast<size_t>(b) * g.max_pages + (r >> g.shift)];
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(g.n_pages)) return -1;
  return ((page * g.Hkv + h) << g.shift) + (r & ((1 << g.shift) - 1));
}

// The same for readers: page 0 in place of a bad one, which is flagged.
__device__ __forceinline__ int paged_row_or_zero(const PagedGeom& g, int b, int h, int r, uint32_t* status) {
  const int y = paged_row(g, b, h, r);
  if (y >= 0) return y;
  if (status) atomicOr(status, EAGLE_STATUS_BAD_PAGE);
  return (h << g.shift) + (r & ((1 << g.shift) - 1));
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The cap in log2 units: c tanh(x) = c - 2 c / (1 + e^2x), in which neither end overflows (e^2x = inf: c, 0: -c); off by
// a few roundings of c, 2e-6 at 30, which a bf16 result does not show.  EXACT (fp32): c tanhf(x), off by a few of itself.
template <bool EXACT = false>
__device__ __forceinline__ float cap_score(const ScoreShape& s, float raw) {
  if (EXACT) return s.cap_log2 * tanhf(raw * s.cap_x);
  return fmaf(-2.f * s.cap_log2, rcp_approx(1.f + sm100::ex2(raw * s.cap_mul)), s.cap_log2);
}

// A raw dot product as a score in log2 units; slope_log2 = slope * log2 e (0: none), dist the row's position minus the
// key's.
template <bool SHAPED, bool EXACT = false>
__device__ __forceinline__ float shape_score(const ScoreShape& s, float raw, float slope_log2, int dist) {
  if (!SHAPED) return raw * s.scale_log2;
  float t = s.cap_log2 > 0.f ? cap_score<EXACT>(s, raw) : raw * s.scale_log2;
  t = fmaf(-slope_log2, static_cast<float>(dist), t);
  return s.window > 0 && dist >= s.window ? -INFINITY : t;
}

// Contiguous bytes (16-byte aligned, a multiple of 16) into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   sm100::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
               : "memory");
}

// sm100::tma_load_3d with an L2 cache policy.
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3, %4}], [%5], %6;" ::"r"(sm100::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(sm100::smem_u32(bar)), "l"(policy)
      : "memory");
}

// Launch with programmatic stream serialization (the kernel waits before it reads or writes); coop: all CTAs resident.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_coop(void (*kern)(KArgs...), bool coop, dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = coop ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              Args... args) {
  return launch_pdl_coop(kern, false, grid, block, smem, s, args...);
}

// Opt-in to `smem` bytes of dynamic shared memory, once per kernel and device.
inline cudaError_t opt_in_smem(const void* kern, int smem, unsigned long long& configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELEASE);
  return e;
}

}  // namespace eagle
