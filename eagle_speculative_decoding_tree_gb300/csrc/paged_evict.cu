// paged_evict.cu -- eviction from a paged cache by accumulated attention weight (eagle_paged_evict).
//
//   select   one CTA per (layer, request, KV head): the `need` heaviest of the rows between the first `sink`
//            and the last `recent`.  Weights become 32-bit keys in the same order; the key of the last one
//            kept is found bit by bit from the top (a radix select: 11, 11 and 10 bits, a histogram in shared
//            memory each), and one more pass writes the kept rows' numbers in order.  The keys stay in shared
//            memory when they fit, so that the weights are read once.
//   move     32 kept rows of K and V a CTA (16 KB in flight) to the request's spare pages.  Out of place:
//            rows need no order among themselves, and what another request shares stays as it is.  The last
//            CTA of a request to finish swaps the pages and sets the length.
// Bound by the kept rows' bytes, read and written once.
#include "paged.cuh"

namespace eagle {
namespace {

constexpr int ST = 512;            // select: threads
constexpr int SW = ST / 32;
constexpr int BINS = 2048;
constexpr int KEYS = 24576;        // keys held in shared memory (96 KB: two CTAs an SM)
constexpr int SELECT_SMEM = KEYS * 4;
constexpr int MT = 256;            // move: threads
constexpr int MR = 32;             // rows a CTA

// Weights as unsigned keys in the same order; NaN is the smallest, both zeros are one.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // (-0 + 0 = 0)
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct EvictArgs {
  PagedGeom g;
  int layers, batch, limit, budget, sink, recent, spare_pages;
  int32_t* table;
  int32_t* spare;
  int32_t* seq_len;
  int32_t* kept;
  uint32_t* status;
  unsigned* count;  // [B] move CTAs done
  unsigned* ready;  // [B] 1: to be moved
};

__device__ __forceinline__ bool evict_over(const EvictArgs& a, int L) { return L > a.limit && L <= a.g.capacity; }

// The bin that holds the `need`-th largest key (counted from the top bin), for all threads; need becomes its
// rank among that bin's keys.
__device__ __forceinline__ int find_bin(const unsigned* hist, int bins, int& need, int* s_scan, int* s_bin) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int per = bins / ST;  // 4 or 2, from the top
  int mine = 0;
  for (int i = 0; i < per; ++i) mine += hist[bins - 1 - (t * per + i)];
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  int before = inc - mine;
  for (int w = 0; w < warp; ++w) before += s_scan[w];
  if (before < need && need <= before + mine) {
    int left = need - before, i = 0;
    for (;; ++i) {
      const int c = hist[bins - 1 - (t * per + i)];
      if (left <= c) break;
      left -= c;
    }
    s_bin[0] = bins - 1 - (t * per + i);
    s_bin[1] = left;
  }
  __syncthreads();
  need = s_bin[1];
  return s_bin[0];
}

__global__ void __launch_bounds__(ST) evict_select_kernel(const EvictArgs a, const PagedEvictArgs p) {
  extern __shared__ uint32_t keys[];
  __shared__ unsigned hist[BINS];
  __shared__ int s_scan[SW], s_bin[2], s_bad, s_gt[SW], s_eq[SW];
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int group = blockIdx.x;  // (l * B + b) * Hkv + h
  const int h = group % a.g.Hkv, lb = group / a.g.Hkv;
  const int b = lb % a.batch, l = lb / a.batch;
  const int L = a.seq_len[b];
  if (!evict_over(a, L)) {
    if (t == 0 && L > a.g.capacity && a.status) atomicOr(a.status, EAGLE_STATUS_CACHE_FULL);
    return;
  }
  if (t == 0) s_bad = 0;
  __syncthreads();
  for (int i = t; i < a.spare_pages; i += ST)
    if (static_cast<unsigned>(a.spare[static_cast<size_t>(b) * a.spare_pages + i]) >= static_cast<unsigned>(a.g.n_pages))
      s_bad = 1;
  __syncthreads();
  if (s_bad) {
    if (t == 0 && a.status) atomicOr(a.status, EAGLE_STATUS_BAD_PAGE);
    return;
  }
  if (t == 0 && l == 0 && h == 0) a.ready[b] = 1;
  int32_t* out = a.kept + static_cast<size_t>(group) * a.budget;
  for (int i = t; i < a.sink; i += ST) out[i] = i;
  for (int i = t; i < a.recent; i += ST) out[a.budget - a.recent + i] = L - a.recent + i;
  const int n = L - a.sink - a.recent;            // candidates (L > limit >= budget >= sink + recent)
  int need = a.budget - a.sink - a.recent;        // of which these stay: need < n
  if (need == 0) return;
  const float* w = p.w[l];
  const bool held = n <= KEYS;
  auto load_key = [&](int i) { return weight_key(w[paged_row_or_zero(a.g, b, h, a.sink + i, a.status)]); };
  auto key_at = [&](int i) { return held ? keys[i] : load_key(i); };
  uint32_t prefix = 0;  // the threshold's bits so far
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass == 2 ? 10 : 11, low = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    for (int i = t; i < BINS; i += ST) hist[i] = 0;
    __syncthreads();
    for (int i = t; i < n; i += ST) {
      uint32_t k;
      if (pass == 0) {
        k = load_key(i);
        if (held) keys[i] = k;
      } else {
        k = key_at(i);
      }
      if (pass == 0 || (k >> (low + bits)) == (prefix >> (low + bits)))
        atomicAdd(&hist[(k >> low) & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    const int bin = find_bin(hist, 1 << bits, need, s_scan, s_bin);
    prefix |= static_cast<uint32_t>(bin) << low;
    __syncthreads();
  }
  // need: how many keys equal to the threshold stay (the lowest rows).  A warp takes a run of candidates.
  const int per = (n + SW - 1) / SW, i0 = min(n, warp * per), i1 = min(n, i0 + per);
  int gt = 0, eq = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = key_at(i);
    gt += k > prefix;
    eq += k == prefix;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  for (int i = 0; i < warp; ++i) {
    gt += s_gt[i];
    eq += s_eq[i];
  }
  const unsigned below = (1u << lane) - 1;
  for (int i = i0; i < i1; i += 32) {
    const int j = i + lane;
    const uint32_t k = j < i1 ? key_at(j) : 0u;
    const bool is_gt = j < i1 && k > prefix, is_eq = j < i1 && k == prefix;
    const unsigned mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq);
    const int e = eq + __popc(me & below);
    if (is_gt || (is_eq && e < need)) out[a.sink + gt + __popc(mg & below) + min(e, need)] = a.sink + j;
    gt += __popc(mg);
    eq += __popc(me);
  }
}

// grid: (layer, request, head) x chunks of MR kept rows.
__global__ void __launch_bounds__(MT) evict_move_kernel(const EvictArgs a, const PagedEvictArgs p, int chunks, int vshift) {
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int t = threadIdx.x;
  const int group = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int h = group % a.g.Hkv, lb = group / a.g.Hkv;
  const int b = lb % a.batch, l = lb / a.batch;
  if (!a.ready[b]) return;
  __shared__ int s_src[MR], s_dst[MR];
  __shared__ bool last;
  const int n0 = chunk * MR, rows = min(MR, a.budget - n0);
  if (t < rows) {
    const int r = a.kept[static_cast<size_t>(group) * a.budget + n0 + t], to = n0 + t;
    const int src = paged_row_or_zero(a.g, b, h, r, a.status);
    const int page = a.spare[static_cast<size_t>(b) * a.spare_pages + (to >> a.g.shift)];
    const int dst = ((page * a.g.Hkv + h) << a.g.shift) + (to & ((1 << a.g.shift) - 1));
    s_src[t] = src;
    s_dst[t] = dst;
    p.w[l][dst] = p.w[l][src];
  }
  __syncthreads();
  const uint4* k = static_cast<const uint4*>(p.k[l]);
  const uint4* v = static_cast<const uint4*>(p.v[l]);
  const int total = rows << vshift, mask = (1 << vshift) - 1;
  constexpr int U = 2;  // (a vector of K and of V each)
  for (int i0 = t; i0 < total; i0 += MT * U) {
    uint4 xk[U], xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * MT;
      if (i < total) {
        const size_t at = (static_cast<size_t>(s_src[i >> vshift]) << vshift) + (i & mask);
        xk[u] = k[at];
        xv[u] = v[at];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * MT;
      if (i < total) {
        const size_t at = (static_cast<size_t>(s_dst[i >> vshift]) << vshift) + (i & mask);
        static_cast<uint4*>(p.k[l])[at] = xk[u];
        static_cast<uint4*>(p.v[l])[at] = xv[u];
      }
    }
  }
  __syncthreads();  // (everyone has the pages)
  if (t == 0) {
    __threadfence();
    const unsigned all = static_cast<unsigned>(a.layers) * a.g.Hkv * chunks;
    last = atomicAdd(&a.count[b], 1u) == all - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int i = t; i < a.spare_pages; i += MT) {
    int32_t* x = a.table + static_cast<size_t>(b) * a.g.max_pages + i;
    int32_t* y = a.spare + static_cast<size_t>(b) * a.spare_pages + i;
    const int32_t old = *x;
    *x = *y;
    *y = old;
  }
  if (t == 0) {
    a.seq_len[b] = a.budget;
    a.count[b] = 0;
    a.ready[b] = 0;
  }
}

}  // namespace

size_t paged_evict_ws(const eagle_paged_evict_desc& d) { return static_cast<size_t>(d.batch) * 8; }

cudaError_t launch_paged_evict(const eagle_paged_evict_desc& d, const PagedEvictArgs& p, int32_t* table,
                               int32_t* spare, int32_t* seq_len, int32_t* kept, uint32_t* status, void* ws,
                               cudaStream_t s) {
  EvictArgs a;
  a.g = paged_geom(table, d.n_pages, d.max_pages, d.page_size, d.n_kv_heads);
  a.layers = d.layers;
  a.batch = d.batch;
  a.limit = d.limit;
  a.budget = d.budget;
  a.sink = d.sink;
  a.recent = d.recent;
  a.spare_pages = (d.budget + d.page_size - 1) / d.page_size;
  a.table = table;
  a.spare = spare;
  a.seq_len = seq_len;
  a.kept = kept;
  a.status = status;
  a.count = static_cast<unsigned*>(ws);
  a.ready = a.count + d.batch;
  static unsigned long long configured = 0;
  cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(evict_select_kernel), SELECT_SMEM, configured);
  if (e != cudaSuccess) return e;
  const int groups = d.layers * d.batch * d.n_kv_heads, chunks = (d.budget + MR - 1) / MR;
  e = launch_pdl(evict_select_kernel, dim3(groups), dim3(ST), SELECT_SMEM, s, a, p);
  if (e != cudaSuccess) return e;
  const int bytes = d.head_dim * (d.dtype == EAGLE_F32 ? 4 : 2);
  return launch_pdl(evict_move_kernel, dim3(static_cast<unsigned>(groups) * chunks), dim3(MT), 0, s, a, p, chunks,
                    bytes == 128 ? 3 : bytes == 256 ? 4 : 5);
}

}  // namespace eagle
