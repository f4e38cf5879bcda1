// paged_weights.cu -- accumulated attention weights of a paged cache's tokens (eagle_paged_weights).
//
// The accepted rows are known only after acceptance, and their softmax sums (lse) since attention: one more
// pass over K gives every key its weight exp(s - lse) without keeping scores.  The keys are divided as the
// attention divides them (paged_attn.cuh); every key belongs to one warp, so nothing is joined and sums have
// a fixed order.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "paged_attn.cuh"
#include "paged_mma.cuh"
#include "tmap.h"

namespace eagle {
namespace {

constexpr int W = 8;   // warps
constexpr int CK = 8;  // keys a warp takes at a time
constexpr int ST = 3;  // ring stages of a warp

struct WeightArgs {
  PagedAttnArgs list;  // the keys of every (request, KV head), one row, no window
  ScoreShape shape;
  const void* q;
  const float* lse;
  const int32_t* n_acc;
  const int32_t* path;
  const float* prior;
  float* weights;
  int R, Hq, G, max_depth;
};

// Path rows of request b (0: the request is left, flagged).  Warp-collective.
__device__ __forceinline__ int path_rows(const WeightArgs& a, int b, int lane) {
  const int na = a.path ? a.n_acc[b] : a.R - 1, L = a.list.seq_len[b];
  bool bad = a.path && (na < 0 || na > a.max_depth);
  if (a.path && !bad)
    for (int m = lane; m <= na; m += 32) {
      const int node = a.path[static_cast<size_t>(b) * (a.max_depth + 1) + m];
      bad |= node < 0 || node >= a.R;
    }
  bad = __any_sync(0xffffffffu, bad);
  const bool full = !bad && (L < na + 1 || L > a.list.g.capacity);
  if (lane == 0 && a.list.status && (bad || full))
    atomicOr(a.list.status, bad ? EAGLE_STATUS_BAD_TREE : EAGLE_STATUS_CACHE_FULL);
  return bad || full ? 0 : na + 1;
}

template <int D, bool SHAPED>
__global__ void __launch_bounds__(W * 32) paged_weights_simt_kernel(const WeightArgs a) {
  using T = float;
  constexpr int N = D / 32, KB = CK * D * sizeof(T);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[W][ST];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * (ST * KB);
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) sm100::mbar_init(&full[warp][i], 1);
    sm100::fence_barrier_init();
  }
  __syncwarp();
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  PagedList list = paged_list(a.list, blockIdx.x, gridDim.x);
  const T* kg = static_cast<const T*>(a.list.k);
  int issued = 0, used = 0;
  bool ok = true;
  while (list.at < list.end && ok) {
    const PagedSegment s = paged_next(a.list, list);
    if (s.t0 >= s.t1) continue;
    const int n = path_rows(a, s.b, lane);
    if (n == 0) continue;
    const int L = s.rq.L, c_end = min(s.t1 * kUnit, L), c0 = s.t0 * kUnit + warp * CK;
    auto issue = [&](int at) {
      if (lane == 0) {
        const size_t y = paged_row_or_zero(a.list.g, s.b, s.h, at, a.list.status);
        sm100::mbar_arrive_expect_tx(&full[warp][issued % ST], KB);
        bulk_load(ring + (issued % ST) * KB, kg + y * D, KB, &full[warp][issued % ST]);
      }
      ++issued;
    };
    int next = c0;
    for (int i = 0; i < ST && next < c_end; ++i, next += W * CK) issue(next);
    const int rows = n * a.G, key = lane & 7;
    for (int at = c0; at < c_end; at += W * CK) {
      const int stage = used % ST;
      ok = __all_sync(0xffffffffu, sm100::wait_parity(&full[warp][stage], (used / ST) & 1, nullptr, 0));
      if (!ok) break;
      ++used;
      const T* ks = reinterpret_cast<const T*>(ring + stage * KB);
      float kx[CK][N];
#pragma unroll
      for (int j = 0; j < CK; ++j) load_part(ks + j * D + lane * N, kx[j]);
      __syncwarp();
      if (next < c_end) {
        issue(next);
        next += W * CK;
      }
      float got = 0.f;
      for (int r0 = 0; r0 < rows; r0 += 4) {
        float x[32];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = min(r0 + r, rows - 1), mm = row / a.G;
          const int node = a.path ? a.path[static_cast<size_t>(s.b) * (a.max_depth + 1) + mm] : mm;
          float q[N];
          load_part(static_cast<const T*>(a.q) +
                        ((static_cast<size_t>(s.b) * a.R + node) * a.Hq + s.h * a.G + row % a.G) * D + lane * N,
                    q);
#pragma unroll
          for (int j = 0; j < CK; ++j) {
            float t = q[0] * kx[j][0];
#pragma unroll
            for (int e = 1; e < N; ++e) t = fmaf(q[e], kx[j][e], t);
            x[r * 8 + j] = t;
          }
        }
        const float raw = spread_sum(x, lane);
        const int row = r0 + (lane >> 3), mm = min(row, rows - 1) / a.G, g = min(row, rows - 1) % a.G;
        const int node = a.path ? a.path[static_cast<size_t>(s.b) * (a.max_depth + 1) + mm] : mm;
        const int dist = L - n + mm - (at + key);
        const float z = a.lse[(static_cast<size_t>(s.b) * a.R + node) * a.Hq + s.h * a.G + g];
        const float slope = SHAPED && a.shape.slopes ? a.shape.slopes[s.h * a.G + g] * kLog2e : 0.f;
        const float t = shape_score<SHAPED, true>(a.shape, raw, slope, dist);
        if (row < rows && dist >= 0 && z != -INFINITY) got += sm100::ex2(t - z * kLog2e);
      }
      got += __shfl_xor_sync(0xffffffffu, got, 8);
      got += __shfl_xor_sync(0xffffffffu, got, 16);
      if (lane < CK && at + key < L) {
        const size_t y = paged_row_or_zero(a.list.g, s.b, s.h, at + key, nullptr);
        const float old = a.prior && at + key < L - n ? a.prior[y] : 0.f;
        if (paged_row(a.list.g, s.b, s.h, at + key) >= 0) a.weights[y] = old + got;
      }
    }
  }
  for (int i = used; i < issued; ++i) (void)sm100::wait_parity(&full[warp][i % ST], (i / ST) & 1, nullptr, 0);
  if (!ok && lane == 0 && a.list.status) atomicOr(a.list.status, EAGLE_STATUS_TIMEOUT);
}

// ---------------------------------------------------------------- bf16
constexpr int MK = 16;  // keys a warp takes at a time
constexpr int MW = 12;  // warps

template <int D>
struct Few {
  static constexpr int KB = MK * D * 2;
  static constexpr int ST = D == 128 ? 4 : 8;  // stages of a warp
  static constexpr int SM_P = MW * ST * KB;     // prior weights, 16 of them a stage
  static constexpr int SM_Y = SM_P + MW * ST * MK * 4;
  static constexpr int SMEM = SM_Y + MW * ST * 4 + 1024;
};

template <int D, int MT, bool SHAPED>
__global__ void __launch_bounds__(MW * 32, 1)
    paged_weights_mma_kernel(const __grid_constant__ CUtensorMap tk, const WeightArgs a) {
  using F = Few<D>;
  constexpr int KS = D / 16, RB = 16 * MT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[MW][F::ST];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qr = lane >> 2, qc = lane & 3;
  uint8_t* ring = smem + warp * (F::ST * F::KB);
  float* sp = reinterpret_cast<float*>(smem + F::SM_P) + warp * (F::ST * MK);
  const uint32_t ring32 = sm100::smem_u32(ring);
  int* sy = reinterpret_cast<int*>(smem + F::SM_Y) + warp * F::ST;  // the stages' rows of the pool, -1: a bad page
  if (lane == 0) {
    sm100::prefetch_tmap(&tk);
    for (int i = 0; i < F::ST; ++i) sm100::mbar_init(&full[warp][i], 1);
    sm100::fence_barrier_init();
  }
  __syncwarp();
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  PagedList list = paged_list(a.list, blockIdx.x, gridDim.x);
  int issued = 0, used = 0;
  bool ok = true;
  const int k_key = ((lane >> 4) << 3) + (lane & 7), k_c = (lane >> 3) & 1;
  while (list.at < list.end && ok) {
    const PagedSegment s = paged_next(a.list, list);
    if (s.t0 >= s.t1) continue;
    const int n = path_rows(a, s.b, lane);
    if (n == 0) continue;
    const int L = s.rq.L, c_end = min(s.t1 * kUnit, L), c0 = s.t0 * kUnit + warp * MK, rows = n * a.G;
    for (int r0 = 0; r0 < rows && ok; r0 += RB) {  // (more than RB rows: what the pass before left is the prior)
      const float* prior = r0 == 0 ? a.prior : a.weights;
      auto issue = [&](int at, int y) {
        if (lane == 0) {
          const int stage = issued % F::ST;
          sy[stage] = y;
          if (y < 0) {  // page 0 in its place, and nothing written
            if (a.list.status) atomicOr(a.list.status, EAGLE_STATUS_BAD_PAGE);
            y = 0;
          }
          uint64_t* bar = &full[warp][stage];
          sm100::mbar_arrive_expect_tx(bar, F::KB + (prior ? MK * 4 : 0));
          sm100::tma_load_3d(ring + stage * F::KB, &tk, 0, y, 0, bar);
          if (prior) bulk_load(sp + stage * MK, prior + y, MK * 4, bar);
        }
        ++issued;
      };
      auto row_of = [&](int at) { return paged_row(a.list.g, s.b, s.h, at); };
      int next = c0, next_row = 0;
      for (int i = 0; i < F::ST && next < c_end; ++i, next += MW * MK) issue(next, lane == 0 ? row_of(next) : 0);
      if (lane == 0 && next < c_end) next_row = row_of(next);
      const bool two = rows - r0 > 16;  // (a short path in a deep tree: the second tile has no rows)
      // the rows: queries, softmax sums (inf: no row), positions
      uint32_t qf[MT][KS][4];
      float z[MT][2], slope[MT][2];
      int pos[MT][2];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = r0 + 16 * t + qr + 8 * i, in = min(row, rows - 1), mm = in / a.G, g = in % a.G;
          const int node = a.path ? a.path[static_cast<size_t>(s.b) * (a.max_depth + 1) + mm] : mm;
          const size_t at = (static_cast<size_t>(s.b) * a.R + node) * a.Hq + s.h * a.G + g;
          const uint16_t* src = static_cast<const uint16_t*>(a.q) + at * D + 2 * qc;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            qf[t][ks][i] = *reinterpret_cast<const uint32_t*>(src + 16 * ks);
            qf[t][ks][i + 2] = *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8);
          }
          const float lse = a.lse[at];
          z[t][i] = row < rows && lse != -INFINITY ? lse * kLog2e : INFINITY;
          slope[t][i] = SHAPED && a.shape.slopes ? a.shape.slopes[s.h * a.G + g] * kLog2e : 0.f;
          pos[t][i] = L - n + mm;
        }
      for (int at = c0; at < c_end; at += MW * MK) {
        const int stage = used % F::ST;
        ok = __all_sync(0xffffffffu, sm100::wait_parity(&full[warp][stage], (used / F::ST) & 1, nullptr, 0));
        if (!ok) break;
        ++used;
        float sc[MT][2][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) sc[t][c][0] = sc[t][c][1] = sc[t][c][2] = sc[t][c][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t b[4];
          const int c = 2 * (ks & 3) + k_c;
          ldsm4(b, ring32 + stage * F::KB + (ks >> 2) * (MK * 128) + k_key * 128 + ((c ^ (k_key & 7)) << 4));
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            if (t && !two) continue;
            mma(sc[t][0], qf[t][ks], b[0], b[1]);
            mma(sc[t][1], qf[t][ks], b[2], b[3]);
          }
        }
        const bool newest = at + MK > L - n;  // some rows do not see some of these keys
        float got[4] = {0.f, 0.f, 0.f, 0.f};  // keys 2 qc, 2 qc + 1, and 8 further on
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (t && !two) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = at + 8 * (e >> 1) + 2 * qc + (e & 1), dist = pos[t][i] - key;
              const float raw = sc[t][e >> 1][2 * i + (e & 1)];
              float x = SHAPED ? shape_score<true>(a.shape, raw, slope[t][i], dist) - z[t][i]
                               : fmaf(raw, a.shape.scale_log2, -z[t][i]);
              if (newest && dist < 0) x = -INFINITY;
              got[e] += sm100::ex2(x);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) got[e] += __shfl_xor_sync(0xffffffffu, got[e], d);
        if (lane < 8) {  // lane: half of the chunk, pair of keys
          const int k = 8 * (lane >> 2) + 2 * (lane & 3);
          const float g0 = lane < 4 ? got[0] : got[2], g1 = lane < 4 ? got[1] : got[3];
          const int y = sy[stage];
          const int old = r0 == 0 ? L - n : L;  // rows whose prior counts
          const float2 p = *reinterpret_cast<const float2*>(sp + stage * MK + k);
          if (y >= 0) {
            if (at + k < L) a.weights[y + k] = (prior && at + k < old ? p.x : 0.f) + g0;
            if (at + k + 1 < L) a.weights[y + k + 1] = (prior && at + k + 1 < old ? p.y : 0.f) + g1;
          }
        }
        __syncwarp();
        if (next < c_end) {
          issue(next, next_row);
          next += MW * MK;
          if (lane == 0 && next < c_end) next_row = row_of(next);
        }
      }
      if (r0 + RB < rows) {  // the next pass's loads go through TMA: what this one wrote must be there
        sm100::fence_proxy_async_global();
        __syncwarp();
      }
    }
  }
  for (int i = used; i < issued; ++i) (void)sm100::wait_parity(&full[warp][i % F::ST], (i / F::ST) & 1, nullptr, 0);
  if (!ok && lane == 0 && a.list.status) atomicOr(a.list.status, EAGLE_STATUS_TIMEOUT);
}

template <int D, int MT, bool SHAPED>
cudaError_t launch_mma(const WeightArgs& a, const CUtensorMap& tk, int ctas, cudaStream_t s) {
  static unsigned long long conf = 0;
  auto kern = paged_weights_mma_kernel<D, MT, SHAPED>;
  constexpr int smem = Few<D>::SMEM;
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, conf);
  return e != cudaSuccess ? e : launch_pdl(kern, dim3(ctas), dim3(MW * 32), smem, s, tk, a);
}

template <int D>
cudaError_t launch_mma_rows(const WeightArgs& a, const CUtensorMap& tk, int rows, bool shaped, int ctas, cudaStream_t s) {
  if (rows <= 16) return shaped ? launch_mma<D, 1, true>(a, tk, ctas, s) : launch_mma<D, 1, false>(a, tk, ctas, s);
  return shaped ? launch_mma<D, 2, true>(a, tk, ctas, s) : launch_mma<D, 2, false>(a, tk, ctas, s);
}

template <int D, bool SHAPED>
cudaError_t launch_simt(const WeightArgs& a, int ctas, cudaStream_t s) {
  static unsigned long long conf = 0;
  auto kern = paged_weights_simt_kernel<D, SHAPED>;
  const int smem = W * ST * CK * D * 4;
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, conf);
  return e != cudaSuccess ? e : launch_pdl(kern, dim3(ctas), dim3(W * 32), smem, s, a);
}

}  // namespace

cudaError_t launch_paged_weights(const eagle_paged_weights_desc& d, const void* q, const float* lse,
                                 const void* k_pages, const int32_t* table, const int32_t* seq_len,
                                 const int32_t* n_acc, const int32_t* path, const float* slopes, const float* prior,
                                 float* weights, uint32_t* status, int sms, cudaStream_t s) {
  WeightArgs a = {};
  a.list.g = paged_geom(table, d.n_pages, d.max_pages, d.page_size, d.n_kv_heads);
  a.list.k = k_pages;
  a.list.seq_len = seq_len;
  a.list.status = status;
  a.list.B = d.batch;
  a.list.R = a.list.G = a.list.rpb = 1;
  a.list.align = a.list.pad = 16;
  a.shape = score_shape(d.scale, d.softcap, d.window, slopes);
  a.q = q;
  a.lse = lse;
  a.n_acc = n_acc;
  a.path = path;
  a.prior = prior;
  a.weights = weights;
  a.R = d.rows;
  a.Hq = d.n_q_heads;
  a.G = d.n_q_heads / d.n_kv_heads;
  a.max_depth = d.max_depth;
  const bool shaped = d.softcap > 0.f || d.window > 0 || slopes;
  if (d.dtype == EAGLE_BF16) {
    CUtensorMap tk;
    if (!make_tmap_halves(&tk, k_pages, d.head_dim, static_cast<unsigned long long>(d.n_pages) * d.n_kv_heads * d.page_size,
                          MK))
      return cudaErrorInvalidValue;
    const int rows = (path ? d.max_depth + 1 : d.rows) * a.G;
    return d.head_dim == 128 ? launch_mma_rows<128>(a, tk, rows, shaped, sms, s)
                             : launch_mma_rows<64>(a, tk, rows, shaped, sms, s);
  }
  const int ctas = 2 * sms;
  if (d.head_dim == 128) return shaped ? launch_simt<128, true>(a, ctas, s) : launch_simt<128, false>(a, ctas, s);
  return shaped ? launch_simt<64, true>(a, ctas, s) : launch_simt<64, false>(a, ctas, s);
}

}  // namespace eagle
