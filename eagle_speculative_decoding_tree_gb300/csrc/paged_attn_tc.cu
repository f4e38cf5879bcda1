// paged_attn_tc.cu -- attention over a paged cache for many query rows of a KV head (draft trees), bf16, head_dim 128,
// on the tcgen05 tensor cores.
//
// Blocks of up to 128 rows against tiles of 128 keys, with the roles and the softmax of tree_attn_tc.cu: a TMA warp, a
// warp that issues S = Q K^T and O += P V, two softmax warpgroups on alternate tiles with states of their own.  What is
// different here:
//   - The keys are divided as in paged_attn.cuh, so a CTA goes through segments; tiles, ring stages and TMEM buffers
//     are counted on through them, and the next segment's loads and first products run under the epilogue of the one
//     before (O is waited for, S and the rings are free).
//     The TMA warp walks the list and leaves the segments for the others in shared memory.
//   - A tile is 128 / T pages, a box of T rows each, found in the page table by the lanes of the TMA warp.
//   - Scores are shaped before the maximum (SHAPED); the window is a range of the tile's keys.
//   - A group's CTAs join their partials together, a share each, after their last segment (one CTA would read 64 KB
//     a partial); the launch is cooperative, every wait bounded.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "attn_tc.cuh"
#include "paged_attn.cuh"
#include "tmap.h"

namespace eagle {
namespace {

using namespace sm100;
using namespace attn_tc;

constexpr int NT = 320;
constexpr int KST = 3, VST = 3;  // ring stages
constexpr int SM_K = TILE;       // behind Q
constexpr int SM_V = SM_K + KST * TILE;
constexpr int SM_ML = SM_V + VST * TILE;  // running maxima and sums [2][128] each
constexpr int SM_DEPTH = SM_ML + 2048;    // the tree keys' depths [128] bytes
constexpr int SM_BAR = SM_DEPTH + 128;
// Segments for the other warps.  The TMA warp writes one when it has loaded the last tile t before it, so QK(t - 3) is
// done, so the softmax has been at tile t - 5 or later: at most 7 segments are in use.
constexpr int SEGS = 8;
constexpr int SM_SEG = SM_BAR + 256;
constexpr int SMEM = SM_SEG + (SEGS + 2) * static_cast<int>(sizeof(PagedSegment));  // two shared ones are kept
constexpr int SMEM_ALLOC = 232448;        // (what is left is room to begin at 1024 bytes)
static_assert(SMEM <= SMEM_ALLOC, "shared memory");
constexpr int RB = 128;                   // rows of a slot

enum : int { ERR_Q = 1, ERR_K = 2, ERR_KE = 4, ERR_V = 8, ERR_VE = 16, ERR_S = 32, ERR_P = 64, ERR_O = 128,
             ERR_GROUP = 256, ERR_QE = 512, ERR_OE = 1024, ERR_SMEM = 2048, ERR_SEG = 4096 };

struct Bars {
  uint64_t q_full, q_empty, k_full[KST], k_empty[KST], v_full[VST], v_empty[VST], s_full[2], p_full[2], o_full, o_free,
      seg_full[SEGS];
  uint32_t tmem_base;
  int go;
};
static_assert(sizeof(Bars) <= 256, "barriers");

struct Maps {
  CUtensorMap q;       // [B R][Hq][128], boxes {64, G, nodes of a block}
  CUtensorMap k, v;    // [pool rows][128], boxes {64, T}
  CUtensorMap tk, tv;  // [B Hkv R][128], boxes {64, 128}
};

__device__ __forceinline__ uint32_t col_s(int j) { return static_cast<uint32_t>(j) * 128u; }
__device__ __forceinline__ uint32_t col_o(int j) { return 256u + static_cast<uint32_t>(j) * 128u; }

// Valid keys of unit u (a tile: the prefix is padded to whole ones).
__device__ __forceinline__ int tile_valid(const PagedAttnArgs& a, const PagedSegment& s, int u) {
  const int at = u * kUnit;
  return at < s.rq.pk ? min(kUnit, s.rq.L - s.rq.k0 - at) : a.tk ? s.rq.Rb : 0;
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 32 raw scores of a row into log2 units; the first key is at distance dist0 (kdepth: tree keys' depths).
__device__ __forceinline__ void shape32(const ScoreShape& sh, uint32_t (&r)[32], float slope, int dist0, int depth,
                                        const int8_t* kdepth) {
  if (sh.cap_log2 > 0.f) {
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < 32; j += 2)
      most = max3(most, fabsf(__uint_as_float(r[j])), fabsf(__uint_as_float(r[j + 1])));
    // Scores well below the cap, the usual case: a polynomial, two scores an instruction (with the formula's two
    // special functions a score 61 rows over 8K took 50 us, so 35).
    if (__all_sync(0xffffffffu, most <= sh.cap_small)) {
      uint64_t p[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) p[i] = f32x2(__float_as_uint(sh.p[i]), __float_as_uint(sh.p[i]));
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const uint64_t x = f32x2(r[j], r[j + 1]), y = mul_f32x2(x, x);
        const uint64_t q = fma_f32x2(y, fma_f32x2(y, fma_f32x2(y, fma_f32x2(y, p[4], p[3]), p[2]), p[1]), p[0]);
        float t0, t1;
        f32x2_split(mul_f32x2(x, q), t0, t1);
        r[j] = __float_as_uint(t0);
        r[j + 1] = __float_as_uint(t1);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(cap_score(sh, __uint_as_float(r[j])));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * sh.scale_log2);
  }
  if (sh.slopes == nullptr) return;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int dist = kdepth ? depth - kdepth[j] : dist0 - j;
    r[j] = __float_as_uint(fmaf(-slope, static_cast<float>(dist), __uint_as_float(r[j])));
  }
}

// This CTA's share of a group's rows from the group's n partials, in pieces of 4 C dims x 32 rows, a warp each: a lane is a
// row.  BATCH partials are in flight together.
template <int BATCH, int C>
__device__ __forceinline__ void join_share(const PagedAttnArgs& a, const PagedSegment& s, int n, int me, int warp, int lane,
                                           int rows) {
  constexpr int U = 128 / C;
  for (int v = U * me / n + warp; v < U * (me + 1) / n; v += 8) {
    const int row = (v & 3) * 32 + lane, c = (v >> 2) * C;
    if (row >= rows) continue;
    float m = -INFINITY, l = 0.f, o[C][4];
#pragma unroll
    for (int k = 0; k < C; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += BATCH) {
      float4 x[BATCH][C];
      float2 ml[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int i = min(i0 + u, n - 1);
        const size_t slot = i == 0 ? s.slot0 : 2 * (s.c0 + i);
        ml[u] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot * RB + row);
#pragma unroll
        for (int k = 0; k < C; ++k) x[u][k] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (slot * 32 + c + k) * RB + row);
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < BATCH; ++u) top = fmaxf(top, ml[u].x);  // (the last one may be there twice)
      const float old = m == -INFINITY ? 0.f : ex2(m - top);
      m = top;
      l *= old;
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][e] *= old;
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        if (i0 + u >= n) continue;
        const float f = ml[u].x == -INFINITY ? 0.f : ex2(ml[u].x - top);
        l = fmaf(f, ml[u].y, l);
#pragma unroll
        for (int k = 0; k < C; ++k) {
          o[k][0] = fmaf(f, x[u][k].x, o[k][0]);
          o[k][1] = fmaf(f, x[u][k].y, o[k][1]);
          o[k][2] = fmaf(f, x[u][k].z, o[k][2]);
          o[k][3] = fmaf(f, x[u][k].w, o[k][3]);
        }
      }
    }
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    const size_t orow = paged_out_row(a, s, s.row0 + row);
    if (a.out_f32) {
#pragma unroll
      for (int k = 0; k < C; ++k)
        reinterpret_cast<float4*>(a.out)[orow * 32 + c + k] =
            make_float4(o[k][0] * inv, o[k][1] * inv, o[k][2] * inv, o[k][3] * inv);
    } else {
      uint32_t w[2 * C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const __nv_bfloat162 t0 = __floats2bfloat162_rn(o[k][0] * inv, o[k][1] * inv);
        const __nv_bfloat162 t1 = __floats2bfloat162_rn(o[k][2] * inv, o[k][3] * inv);
        w[2 * k] = *reinterpret_cast<const uint32_t*>(&t0);
        w[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&t1);
      }
      uint2* dst = reinterpret_cast<uint2*>(a.out) + orow * 32 + c;
      if (C == 1) {
        dst[0] = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int k = 0; k < C; k += 2)
          *reinterpret_cast<uint4*>(dst + k) = make_uint4(w[2 * k], w[2 * k + 1], w[2 * k + 2], w[(2 * k + 3) % (2 * C)]);
      }
    }
    if (a.lse && c == 0) a.lse[orow] = (m + log2f(l)) * 0.69314718055994531f;
  }
}

template <bool PRECISE, bool SHAPED>
__global__ void __launch_bounds__(NT, 1) paged_attn_tc_kernel(const __grid_constant__ Maps tm, const PagedAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (smem - smem_raw > SMEM_ALLOC - SMEM) {  // (not met: the runtime begins it at 1024 bytes)
    if (threadIdx.x == 0) atomicOr(a.err, ERR_SMEM);
    return;
  }
  Bars& bar = *reinterpret_cast<Bars*>(smem + SM_BAR);
  float (*s_m)[128] = reinterpret_cast<float (*)[128]>(smem + SM_ML);
  float (*s_l)[128] = reinterpret_cast<float (*)[128]>(smem + SM_ML + 1024);
  int8_t* s_depth = reinterpret_cast<int8_t*>(smem + SM_DEPTH);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tm.q);
    prefetch_tmap(&tm.k);
    prefetch_tmap(&tm.v);
  }
  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 1);
    for (int i = 0; i < KST; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 128);
    }
    for (int i = 0; i < SEGS; ++i) mbar_init(&bar.seg_full[i], 1);
    mbar_init(&bar.o_full, 1);
    mbar_init(&bar.o_free, 256);
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(&bar.tmem_base, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tb = bar.tmem_base;
  PagedSegment* segs = reinterpret_cast<PagedSegment*>(smem + SM_SEG);
  int tile = 0, seg = 0;  // tiles and segments so far
  bool ok = true;
  // the next segment (NULL: none, or the wait gave up)
  auto next_segment = [&]() -> const PagedSegment* {
    if (!__all_sync(0xffffffffu, wait_parity(&bar.seg_full[seg % SEGS], (seg / SEGS) & 1, a.err, ERR_SEG))) {
      ok = false;
      return nullptr;
    }
    const PagedSegment* s = segs + seg % SEGS;
    return s->t0 < s->t1 ? s : nullptr;
  };

  if (warp == 8) {
    // ------------------------------------------------------------ TMA
    int k_in = 0, v_in = 0, q_in = 0;  // loads issued
    const uint64_t policy = policy_evict_first();  // (what the step reads next stays in L2: the logits, 20 us of a step)
    PagedList list = paged_list(a, blockIdx.x, gridDim.x);
    while (ok) {
      PagedSegment s;
      s.t0 = s.t1 = 0;  // the end
      while (list.at < list.end && s.t0 >= s.t1) s = paged_next(a, list);
      if (lane == 0) {
        segs[seg % SEGS] = s;
        mbar_arrive(&bar.seg_full[seg % SEGS]);
      }
      if (s.t0 >= s.t1) break;
      const int T = 1 << a.g.shift;
      // lane: box lane / 2, half lane % 2 of a tile; its row of the pool (or of the tree), looked up a tile ahead
      auto row_of = [&](int u) {
        const int valid = tile_valid(a, s, u);
        if (u * kUnit >= s.rq.pk) return (s.b * a.g.Hkv + s.h) * a.R;
        return (lane >> 1) << a.g.shift < valid
                   ? paged_row_or_zero(a.g, s.b, s.h, s.rq.k0 + u * kUnit + ((lane >> 1) << a.g.shift), a.status)
                   : 0;
      };
      int y_next = row_of(s.t0);
      for (int u = s.t0; u < s.t1 && ok; ++u, ++tile) {
        const bool tree = u * kUnit >= s.rq.pk;
        const int valid = tile_valid(a, s, u), n = tree ? 1 : (valid + T - 1) >> a.g.shift;  // boxes of a half
        const bool mine = lane < 2 * n && valid > 0;
        const int y = y_next;
        if (u + 1 < s.t1) y_next = row_of(u + 1);
        const int at = (lane & 1) * HALF + (lane >> 1) * T * 128;
        const uint32_t bytes = valid <= 0 ? 0 : tree ? TILE : n * T * 256;
        const int ks = tile % KST, vs = tile % VST;
        if (tile >= KST) ok = __all_sync(0xffffffffu, wait_parity(&bar.k_empty[ks], (tile / KST - 1) & 1, a.err, ERR_KE));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.k_full[ks], bytes);
        ++k_in;
        __syncwarp();
        if (mine)
          tma_load_2d_hint(smem + SM_K + ks * TILE + at, tree ? &tm.tk : &tm.k, 64 * (lane & 1), y, &bar.k_full[ks], policy);
        if (u == s.t0) {  // the rows, behind the first keys
          if (seg > 0) ok = __all_sync(0xffffffffu, wait_parity(&bar.q_empty, (seg - 1) & 1, a.err, ERR_QE));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&bar.q_full, a.rpb * 256);
          ++q_in;
          __syncwarp();
          if (lane < 2)
            tma_load_3d(smem + lane * HALF, &tm.q, 64 * lane, s.h * a.G, s.b * a.R + s.row0 / a.G, &bar.q_full);
        }
        if (tile >= VST) ok = __all_sync(0xffffffffu, wait_parity(&bar.v_empty[vs], (tile / VST - 1) & 1, a.err, ERR_VE));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.v_full[vs], bytes);
        ++v_in;
        __syncwarp();
        if (mine)
          tma_load_2d_hint(smem + SM_V + vs * TILE + at, tree ? &tm.tv : &tm.v, 64 * (lane & 1), y, &bar.v_full[vs], policy);
      }
      ++seg;
    }
    // no copy may still be landing when the CTA ends
    for (int i = 0; i < KST && i < k_in; ++i) (void)wait_parity(&bar.k_full[(k_in - 1 - i) % KST], ((k_in - 1 - i) / KST) & 1, a.err, ERR_K);
    for (int i = 0; i < VST && i < v_in; ++i) (void)wait_parity(&bar.v_full[(v_in - 1 - i) % VST], ((v_in - 1 - i) / VST) & 1, a.err, ERR_V);
    if (q_in > 0) (void)wait_parity(&bar.q_full, (q_in - 1) & 1, a.err, ERR_Q);
  } else if (warp == 9) {
    // ------------------------------------------------------------ products (lane 0)
    while (ok) {
      const PagedSegment* ps = next_segment();
      if (!ps) break;
      const PagedSegment& s = *ps;
      const int n = s.t1 - s.t0;
      auto qk = [&](int i) {  // lane 0
        const int g = tile + i, ks = g % KST;
        if (!wait_parity(&bar.k_full[ks], (g / KST) & 1, a.err, ERR_K)) return false;
        tc_fence_after();
        issue_qk(tb, smem, smem + SM_K + ks * TILE, col_s(g & 1));
        mma_commit(&bar.s_full[g & 1]);
        mma_commit(&bar.k_empty[ks]);
        if (i == n - 1) mma_commit(&bar.q_empty);
        return true;
      };
      if (lane == 0) ok = wait_parity(&bar.q_full, seg & 1, a.err, ERR_Q) && qk(0) && (n < 2 || qk(1));
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      for (int i = 0; i < n && ok; ++i) {
        const int g = tile + i, j = g & 1, vs = g % VST;
        ok = __all_sync(0xffffffffu, wait_parity(&bar.v_full[vs], (g / VST) & 1, a.err, ERR_V));
        if (!ok) break;
        const int nv = max(0, tile_valid(a, s, s.t0 + i));
        if (nv < KT) {  // V rows behind the last key: zeros, whatever they hold
          uint8_t* vt = smem + SM_V + vs * TILE;
          for (int x = lane; x < (KT - nv) * 16; x += 32) {
            const int row = nv + (x >> 4), part = x & 15;
            *reinterpret_cast<uint4*>(vt + (part >> 3) * HALF + row * 128 + (part & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          // O: the segment before has been read
          if (i == 0 && seg > 0) ok = wait_parity(&bar.o_free, (seg - 1) & 1, a.err, ERR_OE);
          ok = ok && wait_parity(&bar.p_full[j], (g >> 1) & 1, a.err, ERR_P);
          if (ok) {
            tc_fence_after();
            issue_pv<PRECISE>(tb, smem + SM_V + vs * TILE, col_s(j), col_o(j), i < 2);
            mma_commit(&bar.v_empty[vs]);
            if (i + 2 < n) ok = qk(i + 2);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      if (lane == 0 && ok) mma_commit(&bar.o_full);
      tile += n;
      ++seg;
    }
  } else {
    // ------------------------------------------------------------ softmax, warps 0-7
    const int wg = warp >> 2, qd = warp & 3, r_local = qd * 32 + lane;
    const uint32_t lb = tb + (static_cast<uint32_t>(qd * 32) << 16);
    const float sl2 = SHAPED ? 1.f : a.shape.scale_log2;
    const uint64_t sl2x2 = f32x2(__float_as_uint(sl2), __float_as_uint(sl2));
    PagedSegment* part = segs + SEGS;  // segments whose group other CTAs share
    int parts = 0;
    for (;;) {
      const PagedSegment* ps = next_segment();
      if (!ps) break;
      const PagedSegment& s = *ps;
      const int n = s.t1 - s.t0;
      const int row = s.row0 + r_local, n_rows = s.rq.Rb * a.G;
      const bool vrow = r_local < a.rpb && row < n_rows;
      const int node = vrow ? row / a.G : 0;
      uint32_t tw[4] = {0u, 0u, 0u, 0u};  // the row's mask words over the tree's keys
      int depth = -1;
      float slope = 0.f;
      if (a.tk && vrow) {
        const uint64_t* w = a.anc_mask + (static_cast<size_t>(s.b) * a.R + node) * a.W;
        const uint64_t w0 = w[0], w1 = a.W > 1 ? w[1] : 0ull;
        tw[0] = static_cast<uint32_t>(w0) & low_bits(s.rq.Rb);
        tw[1] = static_cast<uint32_t>(w0 >> 32) & low_bits(s.rq.Rb - 32);
        tw[2] = static_cast<uint32_t>(w1) & low_bits(s.rq.Rb - 64);
        tw[3] = static_cast<uint32_t>(w1 >> 32) & low_bits(s.rq.Rb - 96);
        depth = max(0, __popc(tw[0]) + __popc(tw[1]) + __popc(tw[2]) + __popc(tw[3]) - 1);
      }
      if (SHAPED) {
        if (a.shape.slopes && vrow) slope = a.shape.slopes[s.h * a.G + row % a.G] * kLog2e;
        if (a.tk && s.t1 * kUnit > s.rq.pk) {
          // (the barrier in the segment before keeps its readers ahead)
          if (threadIdx.x < 128 && static_cast<int>(threadIdx.x) < s.rq.Rb)
            s_depth[threadIdx.x] = static_cast<int8_t>(paged_depth(a, s, threadIdx.x));
          bar_sync(1, 256);
        }
      }
      float m_ref = -INFINITY, l = 0.f;
      for (int i = (tile ^ wg) & 1; i < n; i += 2) {
        const int g = tile + i, u = s.t0 + i;
        ok = __all_sync(0xffffffffu, ok && wait_parity(&bar.s_full[wg], (g >> 1) & 1, a.err, ERR_S));
        if (!ok) break;
        tc_fence_after();
        const bool tree = u * kUnit >= s.rq.pk;
        const int nv = tile_valid(a, s, u);
        const int dist0 = s.rq.L + depth - (s.rq.k0 + u * kUnit);  // to the tile's first key of the prefix
        uint32_t km[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          km[x] = !vrow ? 0u : tree ? tw[x] : low_bits(nv - 32 * x);
          if (SHAPED && !tree && a.shape.window > 0) km[x] &= ~low_bits(dist0 - a.shape.window + 1 - 32 * x);
        }
        if (SHAPED && tree && a.shape.window > 0) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            for (uint32_t left = km[x]; left; left &= left - 1) {
              const int j = __ffs(left) - 1;
              if (depth - s_depth[32 * x + j] >= a.shape.window) km[x] &= ~(1u << j);
            }
        }
        const bool full = __all_sync(0xffffffffu, (km[0] & km[1] & km[2] & km[3]) == 0xffffffffu);
        const uint32_t sc = lb + col_s(wg);
        uint32_t s0[32], s1[32], s2[32], s3[32];
        auto shaped = [&](uint32_t(&r)[32], int x) {
          if (SHAPED) shape32(a.shape, r, slope, dist0 - 32 * x, depth, tree ? s_depth + 32 * x : nullptr);
          if (!full) mask_keys(r, km[x]);
        };
        tmem_ld32(sc, s0);
        tmem_ld32(sc + 32, s1);
        tmem_ld32(sc + 64, s2);
        tmem_ld32(sc + 96, s3);
        tmem_ld_wait();
        shaped(s0, 0);
        shaped(s1, 1);
        if (SHAPED) {  // (they are read again below)
          tmem_st32(sc, s0);
          tmem_st32(sc + 32, s1);
        }
        shaped(s2, 2);
        shaped(s3, 3);
        const float mx = fmaxf(max64(s0, s1), max64(s2, s3));
        const float m_new = fmaxf(m_ref, mx);
        const bool move = m_new != -INFINITY && (m_ref == -INFINITY || (m_new - m_ref) * sl2 > kRescaleLog2);
        const bool scale_o = move && m_ref != -INFINITY;
        const float alpha = scale_o ? ex2((m_ref - m_new) * sl2) : 1.f;
        if (__any_sync(0xffffffffu, scale_o)) {
          l *= alpha;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(lb + col_o(wg) + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(lb + col_o(wg) + 32 * c, o);
          }
          tmem_st_wait();
        }
        if (move) m_ref = m_new;
        const float mu = (m_ref == -INFINITY) ? 0.f : m_ref * sl2;
        const uint64_t nmux2 = f32x2(__float_as_uint(-mu), __float_as_uint(-mu));
        // keys 64..127 first: their P goes where S has been read; keys 0..63 are read again
        float ls = emit_p32<PRECISE>(s2, sc + 64, sl2x2, nmux2);
        ls += emit_p32<PRECISE>(s3, sc + 80, sl2x2, nmux2);
        if (SHAPED) tmem_st_wait();
        tmem_ld32(sc, s0);
        tmem_ld32(sc + 32, s1);
        tmem_ld_wait();
        if (!SHAPED && !full) {
          mask_keys(s0, km[0]);
          mask_keys(s1, km[1]);
        }
        ls += emit_p32<PRECISE>(s0, sc, sl2x2, nmux2);
        ls += emit_p32<PRECISE>(s1, sc + 16, sl2x2, nmux2);
        l += ls;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_full[wg]);
      }
      // ---- the warpgroups' states meet; warpgroup j writes dims [64 j, 64 j + 64) of its row
      ok = __all_sync(0xffffffffu, ok && wait_parity(&bar.o_full, seg & 1, a.err, ERR_O));
      tc_fence_after();
      const float m_own = m_ref * sl2;
      s_m[wg][r_local] = m_own;
      s_l[wg][r_local] = l;
      const bool good = bar_and(1, 256, ok);
      const float mA = s_m[0][r_local], mB = s_m[1][r_local];
      const float M = fmaxf(mA, mB);
      const float fA = mA == -INFINITY ? 0.f : ex2(mA - M), fB = mB == -INFINITY ? 0.f : ex2(mB - M);
      const float L = fmaf(fA, s_l[0][r_local], fB * s_l[1][r_local]);
      // O(j) holds something only if a tile of the segment had that parity
      const bool hasA = n > 1 || (tile & 1) == 0, hasB = n > 1 || (tile & 1) == 1;
      float o[64];
#pragma unroll
      for (int k = 0; k < 64; ++k) o[k] = 0.f;
      if (good) {
        uint32_t x[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (hasA) {
            tmem_ld32(lb + col_o(0) + 64 * wg + 32 * c, x);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[32 * c + k] = fA * __uint_as_float(x[k]);
          }
          if (hasB) {
            tmem_ld32(lb + col_o(1) + 64 * wg + 32 * c, x);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[32 * c + k] = fmaf(fB, __uint_as_float(x[k]), o[32 * c + k]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bar.o_free);
      tile += n;
      const int slot = 2 * blockIdx.x + (seg == 0 ? 0 : 1);
      ++seg;
      if (s.whole()) {
        if (vrow && good) {
          const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
          const size_t orow = paged_out_row(a, s, row);
          if (a.out_f32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * 128 + 64 * wg);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              dst[k] = make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv, o[4 * k + 3] * inv);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * 128 + 64 * wg);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
                w[e] = *reinterpret_cast<const uint32_t*>(&t);
              }
              dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          if (a.lse && wg == 0) a.lse[orow] = (M + log2f(L)) * 0.69314718055994531f;
        }
      } else if (good) {
        if (vrow) {
          // [slot][4 dims][row]: a warp's rows lie together (row by row a CTA's partials took 3.8 us to write)
          float4* dst = reinterpret_cast<float4*>(a.part_o) + (static_cast<size_t>(slot) * 32 + 16 * wg) * RB + r_local;
#pragma unroll
          for (int k = 0; k < 16; ++k) dst[k * RB] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          if (wg == 0)
            *reinterpret_cast<float2*>(a.part_ml + (static_cast<size_t>(slot) * RB + r_local) * 2) = make_float2(M, L);
        }
        __threadfence();
        bar_sync(1, 256);
        if (threadIdx.x == 0) {
          atomicAdd(a.count + s.slot0, 1u);
          part[parts & 1] = s;
        }
        ++parts;
      }
    }
    // ---- shared groups: every CTA joins its share of the rows (all of them are running: cooperative launch)
    bar_sync(1, 256);  // (part)
    for (int i = 0; i < parts; ++i) {
      const PagedSegment s = part[i];
      const int n = s.c1 - s.c0 + 1;
      if (threadIdx.x == 0) bar.go = paged_wait(a, s, ERR_GROUP);
      bar_sync(1, 256);
      const bool go = bar.go != 0;
      bar_sync(1, 256);
      if (!go) continue;
      const int rows = min(a.rpb, s.rq.Rb * a.G - s.row0), me = static_cast<int>(blockIdx.x) - s.c0;
      if (n <= 2)
        join_share<2, 4>(a, s, n, me, warp, lane, rows);
      else if (n <= 4)
        join_share<4, 2>(a, s, n, me, warp, lane, rows);
      else
        join_share<10, 1>(a, s, n, me, warp, lane, rows);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

template <bool PRECISE, bool SHAPED>
cudaError_t launch_tc(const PagedAttnArgs& a, const Maps& tm, int ctas, cudaStream_t s) {
  static unsigned long long conf = 0;
  auto kern = paged_attn_tc_kernel<PRECISE, SHAPED>;
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), SMEM_ALLOC, conf);
  return e != cudaSuccess ? e : launch_pdl_coop(kern, true, dim3(ctas), dim3(NT), SMEM_ALLOC, s, tm, a);
}

}  // namespace

cudaError_t launch_paged_attn_tc(PagedAttnArgs a, int n_pages, bool shaped, bool precise, int ctas, cudaStream_t s) {
  auto fn = tmap_encode_fn();
  if (!fn) return cudaErrorInvalidValue;
  Maps tm;
  const int nodes = 128 / a.G, T = 1 << a.g.shift;
  a.rpb = nodes * a.G;
  a.align = T;
  a.pad = kUnit;
  const unsigned long long pool = static_cast<unsigned long long>(n_pages) * a.g.Hkv * T;
  const unsigned long long tree = static_cast<unsigned long long>(a.B) * a.g.Hkv * a.R;
  constexpr auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr auto SW = CU_TENSOR_MAP_SWIZZLE_128B;
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.B) * a.R};
  const cuuint64_t strides[2] = {256, static_cast<cuuint64_t>(a.Hq) * 256};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(nodes)};
  const cuuint32_t es[3] = {1, 1, 1};
  if (fn(&tm.q, BF, 3, const_cast<void*>(a.q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, SW,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      !make_tmap_2d(&tm.k, BF, 2, a.k, 128, pool, 64, T, SW) || !make_tmap_2d(&tm.v, BF, 2, a.v, 128, pool, 64, T, SW))
    return cudaErrorInvalidValue;
  tm.tk = tm.k;
  tm.tv = tm.v;
  if (a.tk && (!make_tmap_2d(&tm.tk, BF, 2, a.tk, 128, tree, 64, 128, SW) ||
               !make_tmap_2d(&tm.tv, BF, 2, a.tv, 128, tree, 64, 128, SW)))
    return cudaErrorInvalidValue;
  if (shaped) return precise ? launch_tc<true, true>(a, tm, ctas, s) : launch_tc<false, true>(a, tm, ctas, s);
  return precise ? launch_tc<true, false>(a, tm, ctas, s) : launch_tc<false, false>(a, tm, ctas, s);
}

}  // namespace eagle
