// paged_weights.cu -- accumulated attention weights of a paged cache's tokens (eagle_paged_weights).
//
// The accepted rows are known only after acceptance, and their softmax sums (lse) since attention: one more
// pass over K gives every key its weight exp(s - lse) without keeping scores.  The keys are divided as the
// attention divides them (paged_attn.cuh); every key belongs to one warp, so nothing is joined and sums have
// a fixed order.
#include "paged_attn.cuh"

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

template <typename T, int D, bool SHAPED>
__global__ void __launch_bounds__(W * 32) paged_weights_simt_kernel(const WeightArgs a) {
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
  PagedList list = paged_list(a.list, 1, blockIdx.x, gridDim.x);
  const T* kg = static_cast<const T*>(a.list.k);
  int issued = 0, used = 0, err = 0;
  bool ok = true;
  while (list.at < list.end && ok) {
    const PagedSegment s = paged_next(a.list, list, 1);
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
      ok = __all_sync(0xffffffffu, sm100::wait_parity(&full[warp][stage], (used / ST) & 1, &err, 1));
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
        const float t = shape_score<SHAPED>(a.shape, raw, slope, dist);
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
  for (; used < issued; ++used) (void)sm100::wait_parity(&full[warp][used % ST], (used / ST) & 1, &err, 1);
  if (err && a.list.status) atomicOr(a.list.status, EAGLE_STATUS_TIMEOUT);
}

template <typename T, int D, bool SHAPED>
cudaError_t launch_simt(const WeightArgs& a, int ctas, cudaStream_t s) {
  static unsigned long long conf = 0;
  auto kern = paged_weights_simt_kernel<T, D, SHAPED>;
  const int smem = W * ST * CK * D * static_cast<int>(sizeof(T));
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
  a.list.R = a.list.G = 1;
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
  const int ctas = 2 * sms;
  auto run = [&](auto t) {
    using T = decltype(t);
    if (d.head_dim == 128)
      return shaped ? launch_simt<T, 128, true>(a, ctas, s) : launch_simt<T, 128, false>(a, ctas, s);
    return shaped ? launch_simt<T, 64, true>(a, ctas, s) : launch_simt<T, 64, false>(a, ctas, s);
  };
  return d.dtype == EAGLE_F32 ? run(float{}) : run(uint16_t{});
}

}  // namespace eagle
