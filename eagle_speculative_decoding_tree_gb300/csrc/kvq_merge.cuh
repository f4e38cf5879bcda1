// kvq_merge.cuh -- merging a row's partial states (tree attention over the 8-bit cache).
#pragma once

#include "common.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace eagle {

// 128-key tiles of a piece (tcgen05) or units, the tree counted as one, of a split (mma.sync) for
// a request of `tiles` prefix tiles; how many pieces / splits have work.
__device__ __forceinline__ int kvq_tps(const KvqAttnArgs& a, int tiles) {
  if (!a.even) return a.tps;
  return a.tc ? max(1, (tiles + a.splits - 2) / (a.splits - 1)) : (tiles + a.splits) / a.splits;
}
__device__ __forceinline__ int kvq_pieces(const KvqAttnArgs& a, int tiles) {
  const int tps = kvq_tps(a, tiles);
  return min(a.splits, a.tc ? 1 + (tiles + tps - 1) / tps : (tiles + tps) / tps);
}

// The tcgen05 kernels' grid (groups x row blocks, pieces): what this CTA takes.  nrb: row blocks.
__device__ __forceinline__ void kvq_place(const KvqAttnArgs& a, int nrb, int& piece, int& bh, int& rb) {
  int group = blockIdx.x;
  if (a.coop) {
    const int id = blockIdx.y * gridDim.x + blockIdx.x;
    group = id / gridDim.y;
    piece = id % gridDim.y;
  } else {
    piece = blockIdx.y + 1 < gridDim.y ? blockIdx.y + 1 : 0;
  }
  bh = nrb == 1 ? group : group / nrb;
  rb = nrb == 1 ? 0 : group % nrb;
}

// Partial rows come through L2 (other SMs wrote them); volatile, so that the loads of a batch
// stay ahead of everything that uses them.
// Not `on`: zeros, nothing read.
__device__ __forceinline__ void ld_part(const float* p, float (&x)[4], bool on) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n mov.f32 %0, 0f00000000;\n mov.f32 %1, 0f00000000;\n"
      " mov.f32 %2, 0f00000000;\n mov.f32 %3, 0f00000000;\n @q ld.global.cg.v4.f32 {%0,%1,%2,%3}, [%4];\n}\n"
      : "=&f"(x[0]), "=&f"(x[1]), "=&f"(x[2]), "=&f"(x[3])
      : "l"(p), "r"(on ? 1 : 0));
}
__device__ __forceinline__ void ld_part(const float* p, float (&x)[2], bool on) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %3, 0;\n mov.f32 %0, 0f00000000;\n mov.f32 %1, 0f00000000;\n"
      " @q ld.global.cg.v2.f32 {%0,%1}, [%2];\n}\n"
      : "=&f"(x[0]), "=&f"(x[1])
      : "l"(p), "r"(on ? 1 : 0));
}

// The group's meeting under a cooperative launch (every CTA resident).  One thread of a CTA whose
// partials are in place (fenced) counts it in and waits, at most two seconds, until all `need`
// have counted (cnt[0]); past the wait one thread counts it out (cnt[1]), and the last one there
// returns both to zero.
__device__ __forceinline__ bool kvq_group_wait(int* cnt, int need, int* err, int code) {
  atomicAdd(cnt, 1);
  bool all = sm100::ld_acquire_gpu(cnt) >= need;
  if (!all) {
    const uint64_t t0 = sm100::global_ns();
    do {
      __nanosleep(32);
      all = sm100::ld_acquire_gpu(cnt) >= need;
    } while (!all && sm100::global_ns() - t0 < 2000000000ull);
    if (!all) atomicOr(err, code);
  }
  return all;
}
__device__ __forceinline__ void kvq_group_leave(int* cnt, int need) {
  if (atomicAdd(cnt + 1, 1) == need - 1) {
    atomicExch(cnt, 0);
    atomicExch(cnt + 1, 0);
  }
}

// A row's D / 32 dims of this lane, normalised; lane 0 its lse.
template <int D>
__device__ __forceinline__ void kvq_store_row(const KvqAttnArgs& a, size_t orow, int lane, const float (&acc)[D / 32],
                                              float M, float lsum) {
  const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
  const size_t at = orow * D + lane * (D / 32);
#pragma unroll
  for (int e = 0; e < D / 32; e += 2) {
    if (a.out_f32) {
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    } else {
      const __nv_bfloat162 t = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
      *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(a.out) + at + e) = t;
    }
  }
  if (a.lse && lane == 0) a.lse[orow] = (M + log2f(lsum)) * 0.69314718055994531f;
}

// One warp: M = max m_s, out = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s over partials s < n at
// rows base + s rows_pad; D / 32 dims per lane, lane s holds piece s's weight.  BATCH partial rows
// are in flight together (up to 32 pieces a round).  A row with no key gets zeros and lse -inf.
template <int D, int BATCH>
__device__ __forceinline__ void kvq_merge_row(const KvqAttnArgs& a, size_t base, int n, size_t orow, int lane) {
  constexpr int PER = D / 32;
  const float* po = a.part_o + base * D + lane * PER;
  const size_t step = static_cast<size_t>(a.rows_pad);
  float M = -INFINITY, lsum = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < n; s0 += BATCH) {
    float x[BATCH][PER];
    const int mine = s0 + lane;
    const bool has = lane < BATCH && mine < n;
    float ml[2];
    ld_part(a.part_ml + (base + static_cast<size_t>(mine) * step) * 2, ml, has);
#pragma unroll
    for (int u = 0; u < BATCH; ++u) ld_part(po + static_cast<size_t>(s0 + u) * step * D, x[u], s0 + u < n);
    if (!has) ml[0] = -INFINITY;
    const float top = fmaxf(M, warp_max(ml[0]));
    const float old = M == -INFINITY ? 0.f : sm100::ex2(M - top);
    const float f = ml[0] == -INFINITY ? 0.f : sm100::ex2(ml[0] - top);
    M = top;
    lsum = fmaf(lsum, old, warp_sum(f * ml[1]));  // (0 * NaN keeps a poisoned row poisoned)
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= old;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      // no branch on the weight: the loads would sink into it, one after the other
      const float g = __shfl_sync(0xffffffffu, f, u);
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = fmaf(g, x[u][e], acc[e]);
    }
  }
  kvq_store_row<D>(a, orow, lane, acc, M, lsum);
}

// The same for ROWS rows (the first m of them) of at most 16 / ROWS pieces: all their partials are
// in flight together, lane s of the first 16 holds piece s % NP of row s / NP.
template <int D, int ROWS, typename Orow>
__device__ __forceinline__ void kvq_merge_rows(const KvqAttnArgs& a, size_t base, int n, int m, int lane, Orow orow) {
  constexpr int PER = D / 32, NP = 16 / ROWS;
  const float* po = a.part_o + base * D + lane * PER;
  const size_t step = static_cast<size_t>(a.rows_pad);
  const int row = lane / NP, piece = lane % NP;
  const bool has = lane < 16 && row < m && piece < n;
  float ml[2], x[ROWS][NP][PER];
  ld_part(a.part_ml + (base + row + static_cast<size_t>(piece) * step) * 2, ml, has);
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int s = 0; s < NP; ++s)
      ld_part(po + (static_cast<size_t>(s) * step + r) * D, x[r][s], r < m && s < n);
  if (!has) ml[0] = -INFINITY;
  float M = ml[0];
#pragma unroll
  for (int o = NP / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float f = ml[0] == -INFINITY ? 0.f : sm100::ex2(ml[0] - M);
  float lsum = f * ml[1];
#pragma unroll
  for (int o = NP / 2; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    float acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll
    for (int s = 0; s < NP; ++s) {
      const float g = __shfl_sync(0xffffffffu, f, r * NP + s);
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = fmaf(g, x[r][s][e], acc[e]);
    }
    const float Mr = __shfl_sync(0xffffffffu, M, r * NP), lr = __shfl_sync(0xffffffffu, lsum, r * NP);
    if (r < m) kvq_store_row<D>(a, orow(r), lane, acc, Mr, lr);
  }
}

}  // namespace eagle
