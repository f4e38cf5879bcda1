// paged_attn_mma.cu -- attention over a paged cache for few query rows of a KV head (single tokens, chains), bf16, on
// the warp-level matrix instructions.
//
// Few rows against a long cache are bound by the cache's bytes: 16 rows (one instruction's height) need 12 products of
// 16 x 8 x 16 for every 8 keys and 128 dims (K, and V twice for two terms of P), a quarter of what these
// instructions could do in the time that HBM takes to bring the keys.  What has to be avoided is waiting: a warp
// takes 16 keys at a time, K and V by one TMA box each into a ring of its own, and keeps its rows' maxima, sums and
// outputs in registers; warps meet at the end of a segment only (paged_attn.cuh has the division of the keys).
//     S = Q K^T   A = Q, B = K's rows as they lie (ldmatrix)
//     O += P V    A = P, S's registers as they lie, as bf16 (precise: two terms), B = V transposed by ldmatrix
// The exponentials are taken against a reference that moves only when a score is more than 2^kLazy above it, which a
// vote finds out: most chunks need no maximum over the row's lanes.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "paged_attn.cuh"
#include "paged_mma.cuh"
#include "tmap.h"

namespace eagle {
namespace {

constexpr int CK = 16;       // keys
constexpr float kLazy = 8.f; // log2

template <int D, int MT>
struct Few {
  // warps (the registers of D = 128 leave room for 8; half a row is half the bytes a chunk's latency is paid for)
  static constexpr int W = D == 128 ? 8 : 12;
  static constexpr int RB = 16 * MT;                 // rows
  static constexpr int KB = CK * D * 2;              // K of a stage
  static constexpr int ST = D == 128 ? 3 : 4;        // stages of a warp
  static constexpr int RING = ST * 2 * KB;
  static constexpr int LD = D + 8;                   // floats of an output row in shared memory (no bank twice)
  static constexpr int SM_Q = W * RING;              // MT = 2: Q, rows of D, 16-byte chunks swizzled
  static constexpr int SM_M = SM_Q + (MT > 1 ? RB * D * 2 : 0);
  static constexpr int SMEM = SM_M + 2 * W * RB * 4 + 1024;
  static_assert(RB * LD * 4 <= RING, "outputs go where the ring was");
  static_assert(SMEM <= 232448 - 1024, "shared memory");
};

struct Maps {
  CUtensorMap k, v, tk, tv;  // rows of D as [D / 64][rows][64], boxes of 16 rows
};

template <int D, int MT, bool SHAPED, bool PRECISE>
__global__ void __launch_bounds__(Few<D, MT>::W * 32, 1)
    paged_attn_mma_kernel(const __grid_constant__ Maps tm, const PagedAttnArgs a) {
  using F = Few<D, MT>;
  constexpr int W = F::W;
  constexpr int KS = D / 16, NT = D / 8;  // steps of QK's dims, 8-dim tiles of O
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
  // ldmatrix addresses: K chunk (keys, then dims), V chunk (dims, then keys); a half of 64 dims is 16 rows of 128 bytes
  const int k_key = ((lane >> 4) << 3) + (lane & 7), k_c = (lane >> 3) & 1;
  const int v_key = (((lane >> 3) & 1) << 3) + (lane & 7), v_c = lane >> 4;
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
    uint32_t qf[MT == 1 ? KS : 1][4];
    const uint16_t* qg = static_cast<const uint16_t*>(a.q);
    if (MT == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = row0 + qr + 8 * i;
        const uint16_t* src = qg + paged_out_row(a, s, min(row, n_rows - 1)) * D + 2 * qc;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[ks][i] = row < n_rows ? *reinterpret_cast<const uint32_t*>(src + 16 * ks) : 0u;
          qf[ks][i + 2] = row < n_rows ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8) : 0u;
        }
      }
    } else {
      for (int i = threadIdx.x; i < F::RB * (D / 8); i += W * 32) {
        const int r = i / (D / 8), c = i % (D / 8);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row0 + r < n_rows) x = *reinterpret_cast<const uint4*>(qg + paged_out_row(a, s, row0 + r) * D + 8 * c);
        *reinterpret_cast<uint4*>(smem + F::SM_Q + r * (D * 2) + ((c ^ (r & 7)) << 4)) = x;
      }
      __syncthreads();
    }
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
      float sc[MT][2][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < 2; ++n) sc[t][n][0] = sc[t][n][1] = sc[t][n][2] = sc[t][n][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t b[4];
        const int c = 2 * (ks & 3) + k_c;
        ldsm4(b, kb + (ks >> 2) * (CK * 128) + k_key * 128 + ((c ^ (k_key & 7)) << 4));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t af[4];
          if (MT == 1) {
            af[0] = qf[ks][0], af[1] = qf[ks][1], af[2] = qf[ks][2], af[3] = qf[ks][3];
          } else {
            const int r = 16 * t + (lane & 15), qch = 2 * ks + (lane >> 4);
            ldsm4(af, q32 + r * (D * 2) + ((qch ^ (r & 7)) << 4));
          }
          mma(sc[t][0], af, b[0], b[1]);
          mma(sc[t][1], af, b[2], b[3]);
        }
      }
      // ---- scores in log2 units, -inf where hidden
      if (SHAPED || tree || valid < CK) {
        int kd[2][2] = {{0, 0}, {0, 0}};  // depths of the lane's tree keys
        if (SHAPED && tree) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) kd[n][e] = paged_depth(a, s, min(at - pk + 8 * n + 2 * qc + e, a.R - 1));
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t bits = 0xffffu;
            if (tree) {
              const int row = min(row0 + 16 * t + qr + 8 * i, n_rows - 1);
              const uint64_t w = a.anc_mask[(static_cast<size_t>(s.b) * a.R + row / a.G) * a.W + ((at - pk) >> 6)];
              bits = static_cast<uint32_t>(w >> ((at - pk) & 63)) & 0xffffu;
            }
            if (valid < CK) bits &= (1u << valid) - 1;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = 8 * n + 2 * qc + e;
                float& x = sc[t][n][2 * i + e];
                const int dist =
                    tree ? depth[t][i] - kd[n][e] : s.rq.L + depth[t][i] - (s.rq.k0 + at + key);
                if (SHAPED) x = shape_score<true>(a.shape, x, slope[t][i], dist);
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
          const float top = fmaxf(fmaxf(sc[t][0][2 * i], sc[t][0][2 * i + 1]), fmaxf(sc[t][1][2 * i], sc[t][1][2 * i + 1]));
          over |= top * mul > m[t][i] + kLazy;  // (m -inf: any score; -inf never)
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top =
                fmaxf(fmaxf(sc[t][0][2 * i], sc[t][0][2 * i + 1]), fmaxf(sc[t][1][2 * i], sc[t][1][2 * i + 1])) * mul;
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
      uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float neg = m[t][i] == -INFINITY ? 0.f : -m[t][i];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = sm100::ex2(fmaf(sc[t][n][2 * i], mul, neg)), p1 = sm100::ex2(fmaf(sc[t][n][2 * i + 1], mul, neg));
            l[t][i] += p0 + p1;
            const uint32_t h = bf16x2(p0, p1);
            hi[t][2 * n + i] = h;
            if (PRECISE)  // the sum of both terms is off by at most 2^-17 of p
              lo[t][2 * n + i] = bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
          }
        }
      if (valid < CK) {  // V rows behind the last key: zeros, whatever they hold (their p is 0)
        for (int i = lane; i < (CK - valid) * (D / 8); i += 32) {
          const int r = valid + i / (D / 8), c = i % (D / 8);
          *reinterpret_cast<uint4*>(ring + stage * 2 * F::KB + F::KB + (c >> 3) * (CK * 128) + r * 128 + ((c & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        }
        sm100::fence_proxy_async_smem();
        __syncwarp();
      }
      // ---- O
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t b[4];
        const int c = n + v_c;
        ldsm4t(b, vb + (c >> 3) * (CK * 128) + v_key * 128 + (((c & 7) ^ (v_key & 7)) << 4));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          mma(o[t][n], hi[t], b[0], b[1]);
          mma(o[t][n + 1], hi[t], b[2], b[3]);
          if (PRECISE) {
            mma(o[t][n], lo[t], b[0], b[1]);
            mma(o[t][n + 1], lo[t], b[2], b[3]);
          }
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

template <int D, int MT, bool SHAPED, bool PRECISE>
cudaError_t launch_mma(const PagedAttnArgs& a, const Maps& tm, int ctas, cudaStream_t s) {
  static unsigned long long conf = 0;
  auto kern = paged_attn_mma_kernel<D, MT, SHAPED, PRECISE>;
  constexpr int smem = Few<D, MT>::SMEM;
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, conf);
  return e != cudaSuccess ? e : launch_pdl_coop(kern, a.together > 0, dim3(ctas), dim3(Few<D, MT>::W * 32), smem, s, tm, a);
}

template <int D, int MT>
cudaError_t launch_mma_kind(const PagedAttnArgs& a, const Maps& tm, bool shaped, bool precise, int ctas, cudaStream_t s) {
  if (shaped)
    return precise ? launch_mma<D, MT, true, true>(a, tm, ctas, s) : launch_mma<D, MT, true, false>(a, tm, ctas, s);
  return precise ? launch_mma<D, MT, false, true>(a, tm, ctas, s) : launch_mma<D, MT, false, false>(a, tm, ctas, s);
}

}  // namespace

cudaError_t launch_paged_attn_mma(PagedAttnArgs a, int head_dim, long long pool_rows, bool shaped, bool precise,
                                  int ctas, cudaStream_t s) {
  Maps tm;
  const long long tree_rows = static_cast<long long>(a.B) * a.g.Hkv * a.R;
  if (!make_tmap_halves(&tm.k, a.k, head_dim, pool_rows, CK) || !make_tmap_halves(&tm.v, a.v, head_dim, pool_rows, CK))
    return cudaErrorInvalidValue;
  tm.tk = tm.k;
  tm.tv = tm.v;
  if (a.tk && (!make_tmap_halves(&tm.tk, a.tk, head_dim, tree_rows, CK) ||
               !make_tmap_halves(&tm.tv, a.tv, head_dim, tree_rows, CK)))
    return cudaErrorInvalidValue;
  const bool two = a.R * a.G > 16;
  a.rpb = two ? 32 : 16;
  // Groups of so many CTAs share their join (16 heads on one KV head over 12K, 95 CTAs: 20.2 -> 10.4 us; one token of 8
  // heads over 8K, 19 CTAs: 13.6 instead of 13.0; four tokens, 16 rows: 15.9 instead of 16.4).  Only calls of few heads
  // can have such groups, and they alone pay for a cooperative launch.
  const int together = two ? 14 : 20;
  a.together = a.B * a.g.Hkv * together <= ctas ? together : 0;
  if (head_dim == 128)
    return two ? launch_mma_kind<128, 2>(a, tm, shaped, precise, ctas, s)
               : launch_mma_kind<128, 1>(a, tm, shaped, precise, ctas, s);
  return two ? launch_mma_kind<64, 2>(a, tm, shaped, precise, ctas, s)
             : launch_mma_kind<64, 1>(a, tm, shaped, precise, ctas, s);
}

}  // namespace eagle
