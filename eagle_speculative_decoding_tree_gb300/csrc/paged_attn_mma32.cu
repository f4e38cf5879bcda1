// paged_attn_mma32.cu -- attention over a paged cache in fp32 for five query rows of a KV head or more, on the warp-level
// matrix instructions: paged_attn_mma.cu's division of the work, 8 keys a warp at a time.
//
// A product of two fp32 numbers is taken as three of tf32 (11 bits): x = b + s with b = x rounded to tf32 and s the rest,
// and x y = b b + b s + s b, off by 3 2^-22 of |x y| at most (both s rounded, s s left out).  The instructions' own sums
// are cut off, not rounded, so that they are kept short: two steps of a score's dims, one chunk's keys of an output;
// the sums of those are ordinary fp32 additions.  (Products with a small part, 2^-11 of the others, have sums of their own.)
//     S = Q K^T   A = Q from shared memory, B = K's rows as they lie (ldmatrix moves 32-bit elements as well)
//     O += P V    A = P, S's registers as they lie: key 2 c of a lane's column c is the product's key c, 2 c + 1 its c + 4;
//                 B = V, element by element, the same keys
// Bound by the products and by taking the numbers apart: 61 x 4 rows over 4K 114 us, 293 on the ordinary cores.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "paged_attn.cuh"
#include "paged_mma.cuh"
#include "tmap.h"

namespace eagle {
namespace {

constexpr int CK = 8;        // keys
constexpr float kLazy = 8.f; // log2

template <int D, int MT>
struct Few {
  static constexpr int W = 8;                        // warps
  static constexpr int RB = 16 * MT;                 // rows
  static constexpr int KB = CK * D * 4;              // K of a stage
  static constexpr int ST = D == 128 ? 3 : 6;        // stages of a warp
  static constexpr int RING = ST * 2 * KB;
  static constexpr int LD = D + 8;                   // floats of an output row in shared memory (no bank twice)
  static constexpr int SM_Q = W * RING;              // Q, rows of D, 16-byte chunks swizzled
  static constexpr int SM_M = SM_Q + RB * D * 4;
  static constexpr int SMEM = SM_M + 2 * W * RB * 4 + 1024;
  static_assert(RB * LD * 4 <= RING, "outputs go where the ring was");
  static_assert(SMEM <= 232448 - 1024, "shared memory");
};

struct Maps {
  CUtensorMap k, v, tk, tv;  // rows of D as [D / 32][rows][32], boxes of 8 rows
};

// x = big + small, both rounded to tf32 (the instructions ignore the lowest 13 bits of small).
__device__ __forceinline__ void split(float x, uint32_t& big, uint32_t& small) {
  big = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  small = __float_as_uint(x - __uint_as_float(big)) + 0x1000u;
}
__device__ __forceinline__ void mma32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lds(uint32_t addr) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}

template <int D, int MT, bool SHAPED>
__global__ void __launch_bounds__(Few<D, MT>::W * 32, 1)
    paged_attn_mma32_kernel(const __grid_constant__ Maps tm, const PagedAttnArgs a) {
  using F = Few<D, MT>;
  constexpr int W = F::W;
  constexpr int KS = D / 8, NT = D / 8;  // steps of QK's dims, 8-dim tiles of O
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[W][F::ST];
  __shared__ int s_last;
  __shared__ PagedSegment s_part[2];  // segments that are joined together
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qr = lane >> 2, qc = lane & 3;  // a fragment's row and column pair
  uint8_t* ring = smem + warp * F::RING;
  const uint32_t ring32 = sm100::smem_u32(ring), q32 = sm100::smem_u32(smem + F::SM_Q);
  float* s_m = reinterpret_cast<float*>(smem + F::SM_M);
  float* s_l = s_m + W * F::RB;
  if (lane == 0) {
    sm100::prefetch_tmap(&tm.k);
    sm100::prefetch_tmap(&tm.v);
    for (int i = 0; i < F::ST; ++i) sm100::mbar_init(&full[warp][i], 1);
    sm100::fence_barrier_init();
  }
  __syncwarp();
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  PagedList list = paged_list(a, blockIdx.x, gridDim.x);
  const uint64_t policy = sm100::policy_evict_first();
  int issued = 0, used = 0;  // chunks
  int parts = 0;
  bool first = true, ok = true;
  while (list.at < list.end) {
    const PagedSegment s = paged_next(a, list);
    if (s.t0 >= s.t1) continue;
    const int pk = s.rq.pk;
    const int c_end = min(s.t1 * kUnit, pk + (a.tk ? s.rq.Rb : 0)), c0 = s.t0 * kUnit + warp * CK;
    // rows of the pool or of the tree where a chunk begins
    auto row_of = [&](int at) {
      return at < pk ? paged_row_or_zero(a.g, s.b, s.h, s.rq.k0 + at, a.status)
                     : (s.b * a.g.Hkv + s.h) * a.R + (at - pk);
    };
    auto issue = [&](int at, int y) {
      if (lane == 0) {
        uint64_t* bar = &full[warp][issued % F::ST];
        uint8_t* dst = ring + (issued % F::ST) * 2 * F::KB;
        sm100::mbar_arrive_expect_tx(bar, 2 * F::KB);
        tma_load_3d_hint(dst, at < pk ? &tm.k : &tm.tk, 0, y, 0, bar, policy);
        tma_load_3d_hint(dst + F::KB, at < pk ? &tm.v : &tm.tv, 0, y, 0, bar, policy);
      }
      ++issued;
    };
    int next = c0, next_row = 0;
    for (int i = 0; i < F::ST && next < c_end && ok; ++i, next += W * CK) issue(next, lane == 0 ? row_of(next) : 0);
    if (lane == 0 && next < c_end) next_row = row_of(next);  // (on its way while the first chunks are computed)

    // ---- rows
    const int n_rows = s.rq.Rb * a.G, row0 = s.row0;
    const float* qg = static_cast<const float*>(a.q);
    for (int i = threadIdx.x; i < F::RB * (D / 4); i += W * 32) {
      const int r = i / (D / 4), c = i % (D / 4);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row0 + r < n_rows) x = *reinterpret_cast<const uint4*>(qg + paged_out_row(a, s, row0 + r) * D + 4 * c);
      *reinterpret_cast<uint4*>(smem + F::SM_Q + r * (D * 4) + ((c ^ (r & 7)) << 4)) = x;
    }
    __syncthreads();
    float o[MT][NT][4], m[MT][2], l[MT][2], slope[MT][2];
    int depth[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int n = 0; n < NT; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[t][i] = -INFINITY;
        l[t][i] = 0.f;
        const int row = min(row0 + 16 * t + qr + 8 * i, n_rows - 1);
        slope[t][i] = 0.f;
        depth[t][i] = SHAPED && a.tk ? paged_depth(a, s, row / a.G) : -1;
        if (SHAPED && a.shape.slopes) slope[t][i] = a.shape.slopes[s.h * a.G + row % a.G] * kLog2e;
      }
    }

    for (int at = c0; at < c_end; at += W * CK) {
      const int stage = used % F::ST;
      ok = __all_sync(0xffffffffu, ok && sm100::wait_parity(&full[warp][stage], (used / F::ST) & 1, a.err, 1));
      if (!ok) break;
      ++used;
      const uint32_t kb = ring32 + stage * 2 * F::KB, vb = kb + F::KB;
      const bool tree = at >= pk;
      const int valid = tree ? min(CK, s.rq.Rb - (at - pk)) : min(CK, s.rq.L - s.rq.k0 - at);
      // ---- S
      float sc[MT][4];
      float rest[MT][4];  // of the products with a small part
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][e] = rest[t][e] = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < KS; k2 += 2) {
        uint32_t b[4], bb[4], bs[4];  // two steps' K
        const int c = 2 * k2 + (lane >> 3), key = lane & 7;
        ldsm4(b, kb + (c >> 3) * (CK * 128) + key * 128 + (((c & 7) ^ key) << 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) split(__uint_as_float(b[e]), bb[e], bs[e]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = k2; ks < k2 + 2; ++ks) {
            uint32_t q[4], qb[4], qs[4];
            const int r = 16 * t + (lane & 15), qch = 2 * ks + (lane >> 4);
            ldsm4(q, q32 + r * (D * 4) + ((qch ^ (r & 7)) << 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) split(__uint_as_float(q[e]), qb[e], qs[e]);
            const int e = 2 * (ks - k2);
            mma32(rest[t], qs, bb[e], bb[e + 1]);
            mma32(rest[t], qb, bs[e], bs[e + 1]);
            mma32(part, qb, bb[e], bb[e + 1]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][e] += part[e];
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][e] += rest[t][e];
      // ---- scores in log2 units, -inf where hidden
      if (SHAPED || tree || valid < CK) {
        int kd[2] = {0, 0};  // depths of the lane's tree keys
        if (SHAPED && tree) {
#pragma unroll
          for (int e = 0; e < 2; ++e) kd[e] = paged_depth(a, s, min(at - pk + 2 * qc + e, a.R - 1));
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t bits = 0xffu;
            if (tree) {
              const int row = min(row0 + 16 * t + qr + 8 * i, n_rows - 1);
              const uint64_t w = a.anc_mask[(static_cast<size_t>(s.b) * a.R + row / a.G) * a.W + ((at - pk) >> 6)];
              bits = static_cast<uint32_t>(w >> ((at - pk) & 63)) & 0xffu;
            }
            if (valid < CK) bits &= (1u << valid) - 1;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = 2 * qc + e;
              float& x = sc[t][2 * i + e];
              const int dist = tree ? depth[t][i] - kd[e] : s.rq.L + depth[t][i] - (s.rq.k0 + at + key);
              if (SHAPED) x = shape_score<true, true>(a.shape, x, slope[t][i], dist);
              x = (bits >> key) & 1 ? x : -INFINITY;
            }
          }
      }
      const float mul = SHAPED ? 1.f : a.shape.scale_log2;  // (what is left of a score's factor)
      // ---- the reference
      bool over = false;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float top = fmaxf(sc[t][2 * i], sc[t][2 * i + 1]);
          over |= top * mul > m[t][i] + kLazy;  // (m -inf: any score; -inf never)
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(sc[t][2 * i], sc[t][2 * i + 1]) * mul;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            top = fmaxf(top, m[t][i]);
            const float f = m[t][i] == -INFINITY ? 0.f : sm100::ex2(m[t][i] - top);
            m[t][i] = top;
            l[t][i] *= f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              o[t][n][2 * i] *= f;
              o[t][n][2 * i + 1] *= f;
            }
          }
      }
      // ---- P
      uint32_t pb[MT][4], ps[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float neg = m[t][i] == -INFINITY ? 0.f : -m[t][i];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p = sm100::ex2(fmaf(sc[t][2 * i + e], mul, neg));
            l[t][i] += p;
            split(p, pb[t][i + 2 * e], ps[t][i + 2 * e]);
          }
        }
      if (valid < CK) {  // V rows behind the last key: zeros, whatever they hold (their p is 0)
        for (int i = lane; i < (CK - valid) * (D / 4); i += 32) {
          const int r = valid + i / (D / 4), c = i % (D / 4);
          *reinterpret_cast<uint4*>(ring + stage * 2 * F::KB + F::KB + (c >> 3) * (CK * 128) + r * 128 + ((c & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        }
        sm100::fence_proxy_async_smem();
        __syncwarp();
      }
      // ---- O
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = 2 * n + (qr >> 2);
        const uint32_t at0 = vb + (c >> 3) * (CK * 128) + 2 * qc * 128 + (qr & 3) * 4;
        uint32_t b0, b1, s0, s1;
        split(lds(at0 + (((c & 7) ^ (2 * qc)) << 4)), b0, s0);
        split(lds(at0 + 128 + (((c & 7) ^ (2 * qc + 1)) << 4)), b1, s1);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          mma32(part, ps[t], b0, b1);
          mma32(part, pb[t], s0, s1);
          mma32(part, pb[t], b0, b1);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][n][e] += part[e];
        }
      }
      __syncwarp();
      if (next < c_end) {
        issue(next, next_row);
        next += W * CK;
        if (lane == 0 && next < c_end) next_row = row_of(next);
      }
    }

    // ---- the warps' states meet, in the ring (every chunk has been used, or a wait gave up and nothing is valid)
    if (!ok) {
      for (; used < issued; ++used) (void)sm100::wait_parity(&full[warp][used % F::ST], (used / F::ST) & 1, a.err, 1);
    }
    float* so = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[t][i];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        const int r = 16 * t + qr + 8 * i;
        if (qc == 0) {
          s_m[warp * F::RB + r] = m[t][i];
          s_l[warp * F::RB + r] = x;
        }
        if (row0 + r < n_rows) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            *reinterpret_cast<float2*>(so + r * F::LD + 8 * n + 2 * qc) = make_float2(o[t][n][2 * i], o[t][n][2 * i + 1]);
        }
      }
    __syncthreads();
    const bool whole = s.whole();
    const int slot = 2 * blockIdx.x + (first ? 0 : 1);
    for (int r = warp; r < F::RB && row0 + r < n_rows; r += W)
      paged_fold_row<W, F::RB, D>(a, s, whole, slot, r, lane, s_m, s_l, reinterpret_cast<float*>(smem) + r * F::LD,
                                  F::RING / 4);
    sm100::fence_proxy_async_smem();  // the ring is TMA's again
    if (whole) {
      __syncthreads();
    } else if (a.together && s.c1 - s.c0 + 1 >= a.together) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        atomicAdd(a.count + s.slot0, 1u);
        s_part[parts & 1] = s;
      }
      ++parts;
    } else {
      paged_arrive<W, F::RB, D>(a, s, &s_last);
    }
    first = false;
  }
  // ---- long joins: a share of the rows each, a part of the partials a warp
  float* so = reinterpret_cast<float*>(smem);  // [warp][D], the ring is free
  for (int i = 0; i < parts; ++i) {
    __syncthreads();
    const PagedSegment& s = s_part[i];
    if (threadIdx.x == 0) s_last = paged_wait(a, s, 2);
    __syncthreads();
    if (!s_last) continue;
    const int n = s.c1 - s.c0 + 1, me = static_cast<int>(blockIdx.x) - s.c0;
    const int rows = min(F::RB, s.rq.Rb * a.G - s.row0);
    for (int r = rows * me / n; r < rows * (me + 1) / n; ++r) {
      float m, l, o[D / 32];
      paged_join_state<F::RB, D>(a, s, r, lane, n * warp / W, n * (warp + 1) / W, m, l, o);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) so[warp * D + lane * (D / 32) + e] = o[e];
      if (lane == 0) {
        s_m[warp * F::RB + r] = m;
        s_l[warp * F::RB + r] = l;
      }
      __syncthreads();
      if (warp == 0) paged_fold_row<W, F::RB, D>(a, s, true, 0, r, lane, s_m, s_l, so, D);
      __syncthreads();
    }
  }
}

template <int D, int MT, bool SHAPED>
cudaError_t launch_mma32(const PagedAttnArgs& a, const Maps& tm, int ctas, cudaStream_t s) {
  static unsigned long long conf = 0;
  auto kern = paged_attn_mma32_kernel<D, MT, SHAPED>;
  constexpr int smem = Few<D, MT>::SMEM;
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, conf);
  return e != cudaSuccess ? e
                          : launch_pdl_coop(kern, a.together > 0, dim3(ctas), dim3(Few<D, MT>::W * 32), smem, s, tm, a);
}

template <int D, int MT>
cudaError_t launch_mma32_kind(const PagedAttnArgs& a, const Maps& tm, bool shaped, int ctas, cudaStream_t s) {
  return shaped ? launch_mma32<D, MT, true>(a, tm, ctas, s) : launch_mma32<D, MT, false>(a, tm, ctas, s);
}

}  // namespace

cudaError_t launch_paged_attn_mma32(PagedAttnArgs a, int head_dim, long long pool_rows, bool shaped, int ctas,
                                    cudaStream_t s) {
  Maps tm;
  const long long tree_rows = static_cast<long long>(a.B) * a.g.Hkv * a.R;
  if (!make_tmap_halves(&tm.k, a.k, head_dim, pool_rows, CK, 4) || !make_tmap_halves(&tm.v, a.v, head_dim, pool_rows, CK, 4))
    return cudaErrorInvalidValue;
  tm.tk = tm.k;
  tm.tv = tm.v;
  if (a.tk && (!make_tmap_halves(&tm.tk, a.tk, head_dim, tree_rows, CK, 4) ||
               !make_tmap_halves(&tm.tv, a.tv, head_dim, tree_rows, CK, 4)))
    return cudaErrorInvalidValue;
  const bool two = a.R * a.G > 16;
  a.rpb = two ? 32 : 16;
  a.pad = CK;
  const int together = two ? 14 : 20;  // (as paged_attn_mma.cu)
  a.together = a.B * a.g.Hkv * together <= ctas ? together : 0;
  if (head_dim == 128)
    return two ? launch_mma32_kind<128, 2>(a, tm, shaped, ctas, s) : launch_mma32_kind<128, 1>(a, tm, shaped, ctas, s);
  return two ? launch_mma32_kind<64, 2>(a, tm, shaped, ctas, s) : launch_mma32_kind<64, 1>(a, tm, shaped, ctas, s);
}

}  // namespace eagle
