// paged_attn.cu -- attention over a paged cache (eagle_paged_attn): the choice of a kernel, and fp32 for up to four query
// rows of a KV head, on the ordinary cores.
//
// A warp takes 8 keys at a time, of K and of V (one bulk copy each: a page's rows of a head are contiguous),
// in a ring of its own, so that warps meet only at the end of a segment.  Its lanes are the head dims: a lane holds its
// part of four query rows and multiplies 8 keys' parts by them; 32 sums (4 rows x 8 keys) then go to 32 lanes in
// 31 exchanges, each of which halves what a lane has left to sum.  The softmax is that of a lane's score, with the
// running maximum and sum of its row; p goes back to all lanes by shuffles, against V's parts.  Bound by the cache's
// bytes and the exchanges: one token over 32K, 8 KV heads x 128, 50.7 us, 78 % of measured HBM.  (More rows: 16 at a time
// took 293 us for 61 x 4 rows over 4K, paged_attn_mma32.cu 114.)
#include "paged_attn.cuh"

namespace eagle {
namespace {

constexpr int W = 8;    // warps
constexpr int CK = 8;   // keys
constexpr int ST = 3;   // ring stages of a warp

template <int D, int RB>
struct Simt {
  static constexpr int KB = CK * D * 4;             // bytes of a stage's K
  static constexpr int FOLD = RB < 8 ? RB : 8;      // rows folded at a time
  static constexpr int SM_O = W * ST * 2 * KB;
  static constexpr int SM_M = SM_O + W * FOLD * D * 4;
  static constexpr int SMEM = SM_M + 2 * W * RB * 4;
};

template <int D, int RB, bool SHAPED>
__global__ void __launch_bounds__(W * 32, 1) paged_attn_simt_kernel(const PagedAttnArgs a) {
  using S = Simt<D, RB>;
  using T = float;
  constexpr int N = D / 32, RG = RB / 4;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[W][ST];
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* s_o = reinterpret_cast<float*>(smem + S::SM_O);
  float* s_m = reinterpret_cast<float*>(smem + S::SM_M);
  float* s_l = s_m + W * RB;
  uint8_t* ring = smem + warp * (ST * 2 * S::KB);
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) sm100::mbar_init(&full[warp][i], 1);
    sm100::fence_barrier_init();
  }
  __syncwarp();
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  PagedList list = paged_list(a, blockIdx.x, gridDim.x);
  const T* kg = static_cast<const T*>(a.k);
  const T* vg = static_cast<const T*>(a.v);
  int issued = 0, used = 0;  // chunks
  bool first = true, ok = true;
  while (list.at < list.end) {
    const PagedSegment s = paged_next(a, list);
    if (s.t0 >= s.t1) continue;
    const int pk = s.rq.pk;
    const int nk = pk + (a.tk ? s.rq.Rb : 0);
    const int c_end = min(s.t1 * kUnit, nk);
    // this warp's chunks: positions c0, c0 + W CK, ..
    const int c0 = s.t0 * kUnit + warp * CK;
    auto issue = [&](int at) {
      if (lane == 0) {
        const int stage = issued % ST;
        uint8_t* dst = ring + stage * 2 * S::KB;
        const T *ks, *vs;
        uint32_t bytes = S::KB;
        if (at < pk) {
          const size_t y = paged_row_or_zero(a.g, s.b, s.h, s.rq.k0 + at, a.status);
          ks = kg + y * D;
          vs = vg + y * D;
        } else {
          const size_t y = (static_cast<size_t>(s.b) * a.g.Hkv + s.h) * a.R + (at - pk);
          ks = static_cast<const T*>(a.tk) + y * D;
          vs = static_cast<const T*>(a.tv) + y * D;
          bytes = min(CK, a.R - (at - pk)) * D * sizeof(T);
        }
        sm100::mbar_arrive_expect_tx(&full[warp][stage], 2 * bytes);
        bulk_load(dst, ks, bytes, &full[warp][stage]);
        bulk_load(dst + S::KB, vs, bytes, &full[warp][stage]);
      }
      ++issued;
    };
    auto wanted = [&](int at) { return at < c_end && (at >= pk || s.rq.k0 + at < s.rq.L); };
    int next = c0;
    for (int i = 0; i < ST && next < c_end && ok; ++i, next += W * CK)
      if (wanted(next)) issue(next);
    // the rows: a lane's part of q; and as the owner of a score, row lane / 8 of every group of four
    float q[RB][N], o[RB][N], m[RG], l[RG], slope[RG];
    int depth[RG];
    const int n_rows = s.rq.Rb * a.G;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
#pragma unroll
      for (int e = 0; e < N; ++e) q[r][e] = o[r][e] = 0.f;
      if (s.row0 + r < n_rows)
        load_part(static_cast<const T*>(a.q) + paged_out_row(a, s, s.row0 + r) * D + lane * N, q[r]);
    }
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
      const int row = min(s.row0 + 4 * g + (lane >> 3), n_rows - 1);
      slope[g] = a.shape.slopes ? a.shape.slopes[s.h * a.G + row % a.G] * kLog2e : 0.f;
      depth[g] = a.tk ? paged_depth(a, s, row / a.G) : -1;
    }
    for (int at = c0; at < c_end; at += W * CK) {
      if (!wanted(at)) continue;
      const int stage = used % ST;
      ok = __all_sync(0xffffffffu, ok && sm100::wait_parity(&full[warp][stage], (used / ST) & 1, a.err, 1));
      if (!ok) break;
      ++used;
      const T* ks = reinterpret_cast<const T*>(ring + stage * 2 * S::KB);
      const T* vs = ks + CK * D;
      const bool tree = at >= pk;
      const int valid = tree ? min(CK, s.rq.Rb - (at - pk)) : min(CK, s.rq.L - s.rq.k0 - at);
      const int key = lane & 7;
      int kdepth = 0;  // of the lane's tree key
      if (tree && SHAPED && key < valid) {
        kdepth = paged_depth(a, s, at - pk + key);
      }
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        float x[32];
#pragma unroll
        for (int j = 0; j < CK; ++j) {
          float kx[N];
          load_part(ks + j * D + lane * N, kx);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float t = q[4 * g + r][0] * kx[0];
#pragma unroll
            for (int e = 1; e < N; ++e) t = fmaf(q[4 * g + r][e], kx[e], t);
            x[r * 8 + j] = t;
          }
        }
        const float raw = spread_sum(x, lane);
        const int row = s.row0 + 4 * g + (lane >> 3);
        bool on = key < valid && row < n_rows;
        int dist = s.rq.L + depth[g] - (s.rq.k0 + at + key);
        if (tree && on) {
          const uint8_t* bits =
              reinterpret_cast<const uint8_t*>(a.anc_mask + (static_cast<size_t>(s.b) * a.R + row / a.G) * a.W);
          on = (bits[(at - pk) >> 3] >> key) & 1;
          dist = depth[g] - kdepth;
        }
        const float t = on ? shape_score<SHAPED, true>(a.shape, raw, slope[g], dist) : -INFINITY;
        float top = t;
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, m[g]);
        const float alpha = m[g] == -INFINITY ? 0.f : sm100::ex2(m[g] - top);
        const float p = t == -INFINITY ? 0.f : sm100::ex2(t - top);
        if (__any_sync(0xffffffffu, top != m[g])) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float f = __shfl_sync(0xffffffffu, alpha, 8 * r);
#pragma unroll
            for (int e = 0; e < N; ++e) o[4 * g + r][e] *= f;
          }
          l[g] *= alpha;
          m[g] = top;
        }
        l[g] += p;
        for (int j = 0; j < valid; ++j) {
          float vx[N];
          load_part(vs + j * D + lane * N, vx);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float f = __shfl_sync(0xffffffffu, p, 8 * r + j);
            if (f != 0.f) {
#pragma unroll
              for (int e = 0; e < N; ++e) o[4 * g + r][e] = fmaf(f, vx[e], o[4 * g + r][e]);
            }
          }
        }
      }
      __syncwarp();
      while (next < c_end && !wanted(next)) next += W * CK;
      if (next < c_end) {
        issue(next);
        next += W * CK;
      }
    }
    // ---- the warps' states meet
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      float x = l[g];
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if ((lane & 7) == 0) {
        s_m[warp * RB + 4 * g + (lane >> 3)] = m[g];
        s_l[warp * RB + 4 * g + (lane >> 3)] = x;
      }
    }
    const bool whole = s.whole();
    const int slot = 2 * blockIdx.x + (first ? 0 : 1);
#pragma unroll
    for (int f0 = 0; f0 < RB; f0 += S::FOLD) {
#pragma unroll
      for (int r = 0; r < S::FOLD; ++r) {
#pragma unroll
        for (int e = 0; e < N; ++e) s_o[(warp * S::FOLD + r) * D + lane * N + e] = o[f0 + r][e];
      }
      __syncthreads();
      if (warp < S::FOLD)
        paged_fold_row<W, RB, D>(a, s, whole, slot, f0 + warp, lane, s_m, s_l, s_o + warp * D, S::FOLD * D);
      __syncthreads();
    }
    if (!whole) paged_arrive<W, RB, D>(a, s, &s_last);
    first = false;
  }
  // (a wait that gave up: nothing may still be landing)
  for (; used < issued; ++used) (void)sm100::wait_parity(&full[warp][used % ST], (used / ST) & 1, a.err, 1);
}

template <int D, int RB>
cudaError_t launch_simt(PagedAttnArgs a, bool shaped, int ctas, cudaStream_t s) {
  static unsigned long long conf[2] = {0, 0};
  a.rpb = RB;
  auto kern = shaped ? paged_attn_simt_kernel<D, RB, true> : paged_attn_simt_kernel<D, RB, false>;
  const int smem = Simt<D, RB>::SMEM;
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, conf[shaped]);
  return e != cudaSuccess ? e : launch_pdl(kern, dim3(ctas), dim3(W * 32), smem, s, a);
}

constexpr size_t kHead = 256;  // the error word

// Draft trees go to the tensor cores proper, few rows to the kernel that is bound by the cache's bytes.  17 to 32 rows, two
// row tiles there: a chain of 8 x 4 heads over 1K, 8K, 64K and 128K takes 17.4, 25.0, 56.5 and 92.7 us with it, 12.9, 18.3,
// 57 and 100 on tcgen05 (its joins are shared; its softmax is slower than HBM); 16 requests of 0.5K to 9K 84 and 76.5; on
// one KV head (2 x 16 rows over 8K) 11.6 and 15.6.
bool use_tc(const eagle_paged_attn_desc& d) {
  const int G = d.n_q_heads / d.n_kv_heads, rows = d.rows * G;
  if (d.dtype != EAGLE_BF16 || d.head_dim != 128 || G > 128 || d.engine != EAGLE_ENGINE_AUTO) return false;
  return rows > 32 || (rows > 16 && d.batch * d.n_kv_heads >= 4 &&
                       static_cast<long long>(d.max_pages) * d.page_size <= 65536 + 128);
}
size_t slot_rows(const eagle_paged_attn_desc& d) { return use_tc(d) ? 128 : 32; }

}  // namespace

size_t paged_attn_ws(const eagle_paged_attn_desc& d, int sms) {
  const size_t slots = 2 * static_cast<size_t>(sms);
  return kHead + slots * 16 + slots * slot_rows(d) * (static_cast<size_t>(d.head_dim) * 4 + 8);
}

cudaError_t launch_paged_attn(const eagle_paged_attn_desc& d, const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* table, const void* tree_k, const void* tree_v, const int32_t* seq_len,
                              const int32_t* n_nodes, const uint64_t* anc_mask, const float* slopes, void* out,
                              float* lse, uint32_t* status, void* ws, int sms, cudaStream_t s) {
  PagedAttnArgs a;
  a.g = paged_geom(table, d.n_pages, d.max_pages, d.page_size, d.n_kv_heads);
  a.shape = score_shape(d.scale, d.softcap, d.window, slopes);
  a.q = q;
  a.k = k_pages;
  a.v = v_pages;
  a.tk = tree_k;
  a.tv = tree_v;
  a.seq_len = seq_len;
  a.n_nodes = n_nodes;
  a.anc_mask = anc_mask;
  a.out = out;
  a.lse = lse;
  a.status = status;
  const size_t slots = 2 * static_cast<size_t>(sms);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.err = reinterpret_cast<int*>(w);
  a.count = reinterpret_cast<unsigned*>(w + kHead);
  a.leave = a.count + slots;
  a.part_ml = reinterpret_cast<float*>(w + kHead + slots * 16);
  a.part_o = a.part_ml + slots * slot_rows(d) * 2;
  a.B = d.batch;
  a.R = d.rows;
  a.Hq = d.n_q_heads;
  a.G = d.n_q_heads / d.n_kv_heads;
  a.W = (d.rows + 63) / 64;
  a.align = a.pad = 16;
  a.together = 0;
  a.out_f32 = d.out_dtype == EAGLE_F32;
  const bool shaped = d.softcap > 0.f || d.window > 0 || slopes;
  const int rows = d.rows * a.G;
  if (use_tc(d))
    return launch_paged_attn_tc(a, d.n_pages, shaped, d.precision == EAGLE_ATTN_PRECISE, sms, s);
  if (d.dtype == EAGLE_BF16)
    return launch_paged_attn_mma(a, d.head_dim, static_cast<long long>(d.n_pages) * d.n_kv_heads * d.page_size, shaped,
                                 d.precision == EAGLE_ATTN_PRECISE, sms, s);
  if (rows > 4)
    return launch_paged_attn_mma32(a, d.head_dim, static_cast<long long>(d.n_pages) * d.n_kv_heads * d.page_size, shaped,
                                   sms, s);
  return d.head_dim == 128 ? launch_simt<128, 4>(a, shaped, sms, s) : launch_simt<64, 4>(a, shaped, sms, s);
}

}  // namespace eagle
