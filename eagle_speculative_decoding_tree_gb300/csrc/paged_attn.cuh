// paged_attn.cuh -- what the paged attention kernels share: the division of the work and the joining of
// partial results.
//
// The work is a list of units: 128 keys (counted from the first one that any row may see; the tree's own
// keys behind them) of one group, a group being a request, a KV head and a block of query rows.  The groups
// follow one another (request, head, row block), and each CTA takes an even share of the whole list, so that
// ragged lengths need no sorting and no choice of a split: every SM has the same number of keys, whatever the
// requests look like.  A CTA's share covers the end of one group, whole groups, and the beginning of another;
// whole groups are written as they are, of the others the CTA leaves partials (row maxima, sums and
// unnormalised outputs, fp32) in one of its two slots, and the group's last CTA to arrive (a counter) joins
// them, in the order of the list: results do not depend on which one that is.  No CTA waits for another.
#pragma once

#include "paged.cuh"

namespace eagle {

constexpr int kUnit = 128;  // keys

struct PagedAttnArgs {
  PagedGeom g;
  ScoreShape shape;
  const void* q;
  const void* k;
  const void* v;
  const void* tk;  // NULL: no tree
  const void* tv;
  const int32_t* seq_len;
  const int32_t* n_nodes;
  const uint64_t* anc_mask;
  void* out;
  float* lse;
  uint32_t* status;
  int* err;
  unsigned* count;   // [2 CTAs]: arrivals, by the group's first CTA and its slot
  float* part_o;     // [2 CTAs][RB][D]
  float* part_ml;    // [2 CTAs][RB][2]
  int B, R, Hq, G, W;
  int out_f32;
};

// paged_attn_mma.cu: bf16, row blocks of 16 (R G <= 16) or 32.
cudaError_t launch_paged_attn_mma(const PagedAttnArgs& a, int head_dim, long long pool_rows, bool shaped, bool precise,
                                  int ctas, cudaStream_t s);

struct PagedRequest {
  int L, Rb;    // prefix and tree rows
  int k0;       // first key of the list (a multiple of 16)
  int units;    // per group
  int blocks;   // row blocks
};

__device__ __forceinline__ PagedRequest paged_request(const PagedAttnArgs& a, int b, int rows_per_block) {
  PagedRequest r;
  r.L = min(max(a.seq_len[b], 0), a.g.capacity);
  r.Rb = a.n_nodes ? min(max(a.n_nodes[b], 0), a.R) : a.R;
  // the row that stands furthest back is at depth 0, or -1 where its mask is empty
  r.k0 = a.shape.window > 0 ? max(0, r.L - a.shape.window) & ~15 : 0;
  const int keys = ((r.L - r.k0 + 15) & ~15) + (a.tk ? r.Rb : 0);
  r.units = max(1, (keys + kUnit - 1) / kUnit);
  r.blocks = (r.Rb * a.G + rows_per_block - 1) / rows_per_block;
  return r;
}

// A CTA's place in the list.  Every warp keeps its own copy, in step.
struct PagedSegment {
  int b, h, rb;        // group
  PagedRequest rq;
  int t0, t1;          // units of the group
  long long first;     // the group's first unit in the list
};

struct PagedList {
  long long total, at, end;
  int ctas;            // CTAs with work: each has a unit or more
  int b0;              // requests before this one (a multiple of 32) are done
  long long base;      // their units
};

__device__ __forceinline__ long long paged_request_units(const PagedAttnArgs& a, int b, int rows_per_block) {
  if (b >= a.B) return 0;
  const PagedRequest r = paged_request(a, b, rows_per_block);
  return static_cast<long long>(r.units) * r.blocks * a.g.Hkv;
}

__device__ __forceinline__ long long shfl_ll(long long v, int lane) {
  const unsigned lo = __shfl_sync(0xffffffffu, static_cast<unsigned>(v), lane);
  const unsigned hi = __shfl_sync(0xffffffffu, static_cast<unsigned>(static_cast<unsigned long long>(v) >> 32), lane);
  return static_cast<long long>((static_cast<unsigned long long>(hi) << 32) | lo);
}

__device__ __forceinline__ long long list_start(long long total, int cta, int ctas) { return total * cta / ctas; }
// the CTA that has unit u
__device__ __forceinline__ int list_owner(long long total, long long u, int ctas) {
  return static_cast<int>(((u + 1) * ctas - 1) / total);
}

__device__ __forceinline__ PagedList paged_list(const PagedAttnArgs& a, int rows_per_block, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  long long mine = 0;
  for (int b = lane; b < a.B; b += 32) mine += paged_request_units(a, b, rows_per_block);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += shfl_ll(mine, lane ^ o);
  PagedList l;
  l.total = mine;
  l.ctas = static_cast<int>(min(static_cast<long long>(ctas), l.total));
  l.at = l.end = 0;
  if (cta < l.ctas) {
    l.at = list_start(l.total, cta, l.ctas);
    l.end = list_start(l.total, cta + 1, l.ctas);
  }
  l.b0 = 0;
  l.base = 0;
  return l;
}

// The segment at l.at (l.at < l.end); l.at moves behind it.
__device__ __forceinline__ PagedSegment paged_next(const PagedAttnArgs& a, PagedList& l, int rows_per_block) {
  const int lane = threadIdx.x & 31;
  PagedSegment s;
  for (;;) {
    const long long mine = paged_request_units(a, l.b0 + lane, rows_per_block);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = shfl_ll(inc, max(lane - o, 0));
      if (lane >= o) inc += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, l.base + inc > l.at);
    if (past || l.b0 + 32 >= a.B) {
      const int at = past ? __ffs(past) - 1 : 31;
      s.b = min(l.b0 + at, a.B - 1);
      s.first = l.base + shfl_ll(inc - mine, at);
      break;
    }
    l.base += shfl_ll(inc, 31);
    l.b0 += 32;
  }
  s.rq = paged_request(a, s.b, rows_per_block);
  const int group = static_cast<int>((l.at - s.first) / s.rq.units);
  s.first += static_cast<long long>(group) * s.rq.units;
  s.h = group / max(1, s.rq.blocks);
  s.rb = group - s.h * s.rq.blocks;
  s.t0 = static_cast<int>(l.at - s.first);
  s.t1 = static_cast<int>(min(static_cast<long long>(s.rq.units), s.t0 + (l.end - l.at)));
  l.at += s.t1 - s.t0;
  return s;
}

// Where a group's partials are.
struct PagedJoin {
  int c0, c1;  // first and last CTA
  int slot0;   // the first CTA's slot; the others use theirs 0
};
__device__ __forceinline__ PagedJoin paged_join(const PagedList& l, const PagedSegment& s) {
  PagedJoin j;
  j.c0 = list_owner(l.total, s.first, l.ctas);
  j.c1 = list_owner(l.total, s.first + s.rq.units - 1, l.ctas);
  j.slot0 = 2 * j.c0 + (list_start(l.total, j.c0, l.ctas) == s.first ? 0 : 1);
  return j;
}

// A row's place in out ([B][R][Hq] rows) and lse.
__device__ __forceinline__ size_t paged_out_row(const PagedAttnArgs& a, const PagedSegment& s, int row) {
  return (static_cast<size_t>(s.b) * a.R + row / a.G) * a.Hq + s.h * a.G + row % a.G;
}

// N = D / 32 consecutive elements
__device__ __forceinline__ void load_part(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load_part(const float* p, float (&x)[2]) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  x[0] = v.x, x[1] = v.y;
}
// 32 values a lane -> lane i gets the sum over the lanes of value i.
__device__ __forceinline__ float spread_sum(float (&x)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return x[0];
}

// 4 (D = 128) or 2 dims of a row, by one lane of a warp: normalised and stored.
template <int D>
__device__ __forceinline__ void paged_store(const PagedAttnArgs& a, size_t orow, int lane, const float (&o)[D / 32],
                                            float m, float l) {
  constexpr int N = D / 32;
  const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
  const size_t at = orow * D + lane * N;
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    if (a.out_f32) {
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + e) = make_float2(o[e] * inv, o[e + 1] * inv);
    } else {
      const __nv_bfloat162 t = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
      *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(a.out) + at + e) = t;
    }
  }
  if (a.lse && lane == 0) a.lse[orow] = (m + log2f(l)) * 0.69314718055994531f;
}

// One row of a block whose partial state lies in shared memory, W warps' worth: row maxima and sums
// s_m, s_l [W][RB], outputs s_o [W] x `step` floats (the row's).  By one warp.  `whole`: the group is this
// CTA's alone; else into slot `slot`.
template <int W, int RB, int D>
__device__ __forceinline__ void paged_fold_row(const PagedAttnArgs& a, const PagedSegment& s, bool whole, int slot,
                                               int row, int lane, const float* s_m, const float* s_l,
                                               const float* s_o, int step) {
  constexpr int N = D / 32;
  float m = -INFINITY;
#pragma unroll
  for (int w = 0; w < W; ++w) m = fmaxf(m, s_m[w * RB + row]);
  float l = 0.f, o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float mw = s_m[w * RB + row];
    const float f = mw == -INFINITY ? 0.f : sm100::ex2(mw - m);
    l = fmaf(f, s_l[w * RB + row], l);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = fmaf(f, s_o[w * step + lane * N + e], o[e]);
  }
  const int at = s.rb * RB + row;
  if (at >= s.rq.Rb * a.G) return;
  if (whole) {
    paged_store<D>(a, paged_out_row(a, s, at), lane, o, m, l);
  } else {
    float* po = a.part_o + (static_cast<size_t>(slot) * RB + row) * D + lane * N;
#pragma unroll
    for (int e = 0; e < N; e += 2) *reinterpret_cast<float2*>(po + e) = make_float2(o[e], o[e + 1]);
    if (lane == 0)
      *reinterpret_cast<float2*>(a.part_ml + (static_cast<size_t>(slot) * RB + row) * 2) = make_float2(m, l);
  }
}

// A row of a group joined from its CTAs' slots, by one warp.
template <int RB, int D>
__device__ __forceinline__ void paged_join_row(const PagedAttnArgs& a, const PagedSegment& s, const PagedJoin& j,
                                               int row, int lane) {
  constexpr int N = D / 32, BATCH = 8;
  float m = -INFINITY, l = 0.f, o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.f;
  const int n = j.c1 - j.c0 + 1;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int mine = i0 + lane;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (mine < n) {
      const size_t slot = mine == 0 ? j.slot0 : 2 * (j.c0 + mine);
      ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (slot * RB + row) * 2));
    }
    const float top = fmaxf(m, warp_max(ml.x));
    const float old = m == -INFINITY ? 0.f : sm100::ex2(m - top);
    const float f = ml.x == -INFINITY ? 0.f : sm100::ex2(ml.x - top);
    m = top;
    l = fmaf(l, old, warp_sum(f * ml.y));
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] *= old;
    for (int u0 = 0; u0 < 32 && i0 + u0 < n; u0 += BATCH) {
      float2 x[BATCH][N / 2];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int i = min(i0 + u0 + u, n - 1);
        const size_t slot = i == 0 ? j.slot0 : 2 * (j.c0 + i);
        const float* po = a.part_o + (slot * RB + row) * D + lane * N;
#pragma unroll
        for (int e = 0; e < N / 2; ++e) x[u][e] = __ldcg(reinterpret_cast<const float2*>(po) + e);
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const float g = __shfl_sync(0xffffffffu, f, (u0 + u) & 31);
        if (i0 + u0 + u < n) {
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            o[2 * e] = fmaf(g, x[u][e].x, o[2 * e]);
            o[2 * e + 1] = fmaf(g, x[u][e].y, o[2 * e + 1]);
          }
        }
      }
    }
  }
  paged_store<D>(a, paged_out_row(a, s, s.rb * RB + row), lane, o, m, l);
}

// The end of a segment whose group other CTAs share: this CTA's partials are written; the last CTA of the
// group joins them.  By all W warps of the CTA (barrier 0).
template <int W, int RB, int D>
__device__ __forceinline__ void paged_arrive(const PagedAttnArgs& a, const PagedList& l, const PagedSegment& s,
                                             int* s_last) {
  const PagedJoin j = paged_join(l, s);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned n = j.c1 - j.c0 + 1;
    const bool last = atomicAdd(a.count + j.slot0, 1u) == n - 1;
    if (last) a.count[j.slot0] = 0;
    __threadfence();
    *s_last = last;
  }
  __syncthreads();
  if (!*s_last) return;
  const int rows = min(RB, s.rq.Rb * a.G - s.rb * RB);
  for (int row = threadIdx.x >> 5; row < rows; row += W) paged_join_row<RB, D>(a, s, j, row, threadIdx.x & 31);
}

}  // namespace eagle
