// paged_attn.cuh -- what the paged attention kernels share: the division of the work and the joining of
// partial results.
//
// The work is a list of units: 128 keys (counted from the first one that any row may see; the tree's own
// keys behind them) of one group, a group being a request, a KV head and a block of query rows.  The groups
// follow one another (row block, request, head: so that the row blocks of a head, which read the same keys, are
// at work at the same time and share them through L2: one CTA after the other asked HBM for a tile of 64 KB every
// 1.7 us an SM, 5.8 TB/s), and each CTA takes an even share of the whole list, so that
// ragged lengths need no sorting and no choice of a split: every SM has the same number of keys, whatever the
// requests look like.  A CTA's share covers the end of one group, whole groups, and the beginning of another;
// whole groups are written as they are, of the others the CTA leaves partials (row maxima, sums and
// unnormalised outputs, fp32) in one of its two slots, and the group's last CTA to arrive (a counter) joins
// them, in the order of the list: results do not depend on which one that is.  No CTA waits for another, but where a
// join is so long that its CTAs share it (`together`, a cooperative launch).
// With kSplitFrom CTAs a group or more, shares end with the groups: each group has CTAs in proportion to its
// units, and a CTA one segment (one token over 8K 15.8 -> 13.0 us, 61 rows 32.5 -> 24.7; 4 requests of 61 rows, two CTAs a
// group, which stay with even shares: 62.7 and 63.0).
#pragma once

#include "paged.cuh"

namespace eagle {

constexpr int kUnit = 128;    // keys
constexpr int kSplitFrom = 3; // CTAs a group from which each CTA has a part of one group only

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
  unsigned* leave;   // [2 CTAs]: CTAs past their wait, where they wait
  float* part_o;     // [2 CTAs][RB][D]
  float* part_ml;    // [2 CTAs][RB][2]
  int B, R, Hq, G, W;
  int rpb;           // rows of a block
  int align, pad;    // the list's first key and the prefix's positions are multiples of these
  int out_f32;
  int together;      // from this many CTAs a group on, they join their partials together (0: never)
};

// paged_attn_mma.cu: bf16, row blocks of 16 (R G <= 16) or 32.
cudaError_t launch_paged_attn_mma(PagedAttnArgs a, int head_dim, long long pool_rows, bool shaped, bool precise,
                                  int ctas, cudaStream_t s);
// paged_attn_mma32.cu: fp32, row blocks as above.
cudaError_t launch_paged_attn_mma32(PagedAttnArgs a, int head_dim, long long pool_rows, bool shaped, int ctas,
                                    cudaStream_t s);
// paged_attn_tc.cu: bf16, head_dim 128, G <= 128, row blocks of 128 / G nodes.
cudaError_t launch_paged_attn_tc(PagedAttnArgs a, int n_pages, bool shaped, bool precise, int ctas, cudaStream_t s);

struct PagedRequest {
  int L, Rb;    // prefix and tree rows
  int k0;       // first key of the list
  int pk;       // list positions of the prefix (the tree's keys come behind them)
  int units;    // per group
  int blocks;   // row blocks
};

__device__ __forceinline__ PagedRequest paged_request(const PagedAttnArgs& a, int b) {
  PagedRequest r;
  r.L = min(max(a.seq_len[b], 0), a.g.capacity);
  r.Rb = a.n_nodes ? min(max(a.n_nodes[b], 0), a.R) : a.R;
  // the row that stands furthest back is at depth 0 (without a tree: -1)
  r.k0 = a.shape.window > 0 ? max(0, r.L - a.shape.window + (a.tk ? 1 : 0)) & ~(a.align - 1) : 0;
  r.pk = (r.L - r.k0 + a.pad - 1) & ~(a.pad - 1);
  r.units = max(1, (r.pk + (a.tk ? r.Rb : 0) + kUnit - 1) / kUnit);
  r.blocks = (r.Rb * a.G + a.rpb - 1) / a.rpb;
  return r;
}

// A part of a group that one CTA takes.
struct PagedSegment {
  int b, h, row0;      // group; its first row
  PagedRequest rq;
  int t0, t1;          // units of the group
  int c0, c1;          // the group's first and last CTA
  int slot0;           // the first CTA's slot; the others use theirs 0
  __device__ bool whole() const { return t0 == 0 && t1 == rq.units; }
};

// A CTA's place in the list.  Every warp keeps its own copy, in step.  (Counts of units are 32-bit: the entry points
// refuse more.)
struct PagedList {
  int total, groups;   // units, groups
  int ctas;            // CTAs with work: each a unit or more
  int per, more;       // units a CTA, and how many CTAs have one more
  bool split;          // each CTA has a part of one group
  unsigned pace;       // split: CTAs a unit, 0.32 fixed point, behind one a group
  int at, end;         // units (split: at = the CTA, end = at + 1)
  int plane;           // row block
  int b0;              // requests before this one (a multiple of 32) are done:
  int base, gbase;     // their units and groups
  int inc, ginc;       // the lane's request b0 + lane: units and groups up to it, from b0 on
};

__device__ __forceinline__ int list_start(const PagedList& l, int cta) { return cta * l.per + min(cta, l.more); }
// the CTA that has unit u
__device__ __forceinline__ int list_owner(const PagedList& l, int u) {
  const int k = l.more * (l.per + 1);
  return u < k ? u / (l.per + 1) : l.more + (u - k) / l.per;
}
// split: the first CTA of group g, whose first unit is u: one a group, the others by units
__device__ __forceinline__ int split_start(const PagedList& l, int g, int u) {
  return g + min(static_cast<int>(__umulhi(static_cast<unsigned>(u), l.pace)), l.ctas - l.groups);
}

// inc, ginc of the 32 requests from l.b0 on, of row block l.plane
__device__ __forceinline__ void list_scan(const PagedAttnArgs& a, PagedList& l) {
  const int lane = threadIdx.x & 31;
  l.inc = l.ginc = 0;
  if (l.b0 + lane < a.B) {
    const PagedRequest r = paged_request(a, l.b0 + lane);
    l.ginc = r.blocks > l.plane ? a.g.Hkv : 0;
    l.inc = r.units * l.ginc;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, l.inc, o), y = __shfl_up_sync(0xffffffffu, l.ginc, o);
    if (lane >= o) {
      l.inc += x;
      l.ginc += y;
    }
  }
}

__device__ __forceinline__ PagedList paged_list(const PagedAttnArgs& a, int cta, int ctas) {
  PagedList l;
  l.total = l.groups = l.plane = 0;
  l.b0 = l.base = l.gbase = 0;
  if (a.B <= 32 && a.R * a.G <= a.rpb) {  // (the common case: one scan does)
    list_scan(a, l);
    l.total = __shfl_sync(0xffffffffu, l.inc, 31);
    l.groups = __shfl_sync(0xffffffffu, l.ginc, 31);
  } else {
#pragma unroll 4
    for (int b = threadIdx.x & 31; b < a.B; b += 32) {
      const PagedRequest r = paged_request(a, b);
      l.groups += r.blocks * a.g.Hkv;
      l.total += r.units * r.blocks * a.g.Hkv;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      l.groups += __shfl_xor_sync(0xffffffffu, l.groups, o);
      l.total += __shfl_xor_sync(0xffffffffu, l.total, o);
    }
    list_scan(a, l);
  }
  l.ctas = min(ctas, l.total);
  l.split = l.groups * kSplitFrom <= l.ctas;
  l.per = l.more = l.at = l.end = 0;
  l.pace = 0;
  if (cta >= l.ctas) return l;
  if (l.split) {
    // a little above (ctas - groups) / total 2^32: equal groups get equal numbers
    l.pace = static_cast<unsigned>(static_cast<float>(l.ctas - l.groups) / static_cast<float>(l.total) * 4294972000.f);
    l.at = cta;
    l.end = cta + 1;
  } else {
    l.per = l.total / l.ctas;
    l.more = l.total - l.per * l.ctas;
    l.at = list_start(l, cta);
    l.end = list_start(l, cta + 1);
  }
  return l;
}

// The segment at l.at (l.at < l.end); l.at moves behind it.  It may be empty (t0 = t1).
__device__ __forceinline__ PagedSegment paged_next(const PagedAttnArgs& a, PagedList& l) {
  PagedSegment s;
  int first, g, prev, gprev;  // the request's first unit and group
  for (;;) {
    const int past = l.split ? split_start(l, l.gbase + l.ginc, l.base + l.inc) : l.base + l.inc;
    const unsigned m = __ballot_sync(0xffffffffu, past > l.at);
    const bool last = l.b0 + 32 >= a.B && (l.plane + 1) * a.rpb >= a.R * a.G;
    if (m || last) {
      // (split: a CTA behind the last group's is given that group, and finds nothing there)
      int at = m ? __ffs(m) - 1 : 31;
      if (!m) at = __ffs(__ballot_sync(0xffffffffu, l.ginc == __shfl_sync(0xffffffffu, l.ginc, 31))) - 1;
      prev = __shfl_sync(0xffffffffu, l.inc, max(at - 1, 0));
      gprev = __shfl_sync(0xffffffffu, l.ginc, max(at - 1, 0));
      s.b = l.b0 + at;
      first = l.base + (at ? prev : 0);
      g = l.gbase + (at ? gprev : 0);
      break;
    }
    l.base += __shfl_sync(0xffffffffu, l.inc, 31);
    l.gbase += __shfl_sync(0xffffffffu, l.ginc, 31);
    l.b0 += 32;
    if (l.b0 >= a.B) {
      l.b0 = 0;
      ++l.plane;
    }
    list_scan(a, l);
  }
  s.rq = paged_request(a, s.b);
  const int n = s.rq.units;
  int i;  // head
  if (s.rq.blocks <= l.plane) {  // (the last requests have no such rows, and the CTA is behind the last group's)
    s.h = s.row0 = s.t0 = s.t1 = s.c0 = s.c1 = s.slot0 = 0;
    l.at = l.end;
    return s;
  }
  if (l.split) {
    int lo = 0, hi = a.g.Hkv - 1;  // the last one that starts at this CTA or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (split_start(l, g + mid, first + mid * n) <= l.at)
        lo = mid;
      else
        hi = mid - 1;
    }
    i = lo;
    first += i * n;
    s.c0 = split_start(l, g + i, first);
    s.c1 = split_start(l, g + i + 1, first + n) - 1;
    s.slot0 = 2 * s.c0;
    // (a group of fewer units than CTAs: some have none, and nothing to leave)
    const int k = min(s.c1 - s.c0 + 1, n), j = l.at - s.c0;
    s.c1 = s.c0 + k - 1;
    const int q = n / k, r = n - q * k;
    s.t0 = j < k ? j * q + min(j, r) : n;
    s.t1 = j < k ? s.t0 + q + (j < r ? 1 : 0) : n;
    l.at = l.end;
  } else {
    i = (l.at - first) / n;
    first += i * n;
    s.t0 = l.at - first;
    s.t1 = min(n, s.t0 + (l.end - l.at));
    l.at += s.t1 - s.t0;
    s.c0 = list_owner(l, first);
    s.c1 = list_owner(l, first + n - 1);
    s.slot0 = 2 * s.c0 + (list_start(l, s.c0) == first ? 0 : 1);
  }
  s.h = i;
  s.row0 = l.plane * a.rpb;
  return s;
}

// How far a tree node stands behind the prefix: the bits of its mask row among the request's nodes, less one.
__device__ __forceinline__ int paged_depth(const PagedAttnArgs& a, const PagedSegment& s, int node) {
  const uint64_t* w = a.anc_mask + (static_cast<size_t>(s.b) * a.R + node) * a.W;
  int c = 0;
  for (int i = 0; i < a.W; ++i) {
    const int live = s.rq.Rb - 64 * i;
    c += __popcll(live >= 64 ? w[i] : live > 0 ? w[i] & ((1ull << live) - 1) : 0ull);
  }
  return max(c - 1, 0);
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
  const int at = s.row0 + row;
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

// A row's state from slots i0 .. i1 - 1 of its group, by one warp.  The partial rows of BATCH CTAs are requested before
// their weights are known.
template <int RB, int D>
__device__ __forceinline__ void paged_join_state(const PagedAttnArgs& a, const PagedSegment& s, int row, int lane, int i0,
                                                 int i1, float& m, float& l, float (&o)[D / 32]) {
  constexpr int N = D / 32, BATCH = 20;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.f;
  auto place = [&](int i) { return static_cast<size_t>(i == 0 ? s.slot0 : 2 * (s.c0 + i)) * RB + row; };
#pragma unroll 1
  for (; i0 < i1; i0 += BATCH) {
    float2 x[BATCH][N / 2], ml = make_float2(-INFINITY, 0.f);
    const int mine = i0 + lane;
    if (lane < BATCH && mine < i1) ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + place(mine));
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const float2* po = reinterpret_cast<const float2*>(a.part_o + place(min(i0 + u, i1 - 1)) * D + lane * N);
#pragma unroll
      for (int e = 0; e < N / 2; ++e) x[u][e] = __ldcg(po + e);
    }
    const float top = fmaxf(m, warp_max(ml.x));
    const float old = m == -INFINITY ? 0.f : sm100::ex2(m - top);
    const float f = ml.x == -INFINITY ? 0.f : sm100::ex2(ml.x - top);
    m = top;
    l = fmaf(l, old, warp_sum(f * ml.y));
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] *= old;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const float g = __shfl_sync(0xffffffffu, f, u);
      if (i0 + u < i1) {  // (the others' row is there twice)
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          o[2 * e] = fmaf(g, x[u][e].x, o[2 * e]);
          o[2 * e + 1] = fmaf(g, x[u][e].y, o[2 * e + 1]);
        }
      }
    }
  }
}

// The end of a segment whose group other CTAs share: this CTA's partials are written; the last CTA of the
// group joins them.  By all W warps of the CTA (barrier 0).
template <int W, int RB, int D>
__device__ __forceinline__ void paged_arrive(const PagedAttnArgs& a, const PagedSegment& s, int* s_last) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned n = s.c1 - s.c0 + 1;
    const bool last = atomicAdd(a.count + s.slot0, 1u) == n - 1;
    if (last) a.count[s.slot0] = 0;
    __threadfence();
    *s_last = last;
  }
  __syncthreads();
  if (!*s_last) return;
  const int rows = min(RB, s.rq.Rb * a.G - s.row0);
  for (int row = threadIdx.x >> 5; row < rows; row += W) {
    float m, l, o[D / 32];
    paged_join_state<RB, D>(a, s, row, threadIdx.x & 31, 0, s.c1 - s.c0 + 1, m, l, o);
    paged_store<D>(a, paged_out_row(a, s, s.row0 + row), threadIdx.x & 31, o, m, l);
  }
}

// Waits (one thread; cooperative launch) until the group's CTAs have left their partials; the last one past it returns
// the counters to zero.
__device__ __forceinline__ bool paged_wait(const PagedAttnArgs& a, const PagedSegment& s, int err) {
  const int n = s.c1 - s.c0 + 1;
  const int* count = reinterpret_cast<const int*>(a.count + s.slot0);
  bool all = sm100::ld_acquire_gpu(count) >= n;
  const uint64_t t0 = sm100::global_ns();
  while (!all && sm100::global_ns() - t0 < 2000000000ull) {
    __nanosleep(32);
    all = sm100::ld_acquire_gpu(count) >= n;
  }
  if (!all) {
    atomicOr(a.err, err);
    return false;
  }
  if (atomicAdd(a.leave + s.slot0, 1u) == static_cast<unsigned>(n) - 1) {
    atomicExch(a.count + s.slot0, 0u);
    atomicExch(a.leave + s.slot0, 0u);
  }
  return true;
}

}  // namespace eagle
