// paged_evict.cu -- eviction from a paged cache by accumulated attention weight (eagle_paged_evict).
//
//   select   one CTA per (request, layer, KV head): the `need` heaviest of the rows between the first `sink`
//            and the last `recent`.  Weights become 32-bit keys in the same order; the key of the last one
//            kept is found from the top (a radix select: 11, 11 and 10 bits, a histogram in shared memory
//            each), and one more pass writes the kept rows' numbers in order.  The keys stay in shared memory
//            when they fit, so that the weights are read once, four a load and all loads of a thread together.
//   move     each CTA takes an even share of all requests' pieces of 64 kept rows.  One warp looks the next
//            piece's rows up (three loads that wait for one another) and moves their weights, the others copy
//            K and V, 64 bytes a thread in flight.  Out of place, to the request's spare pages: rows need no
//            order among themselves, and what another request shares stays as it is.  The last CTA of a request to finish swaps the pages and sets the length.
// Bound by the kept rows' bytes, read and written once.
#include "paged.cuh"

namespace eagle {
namespace {

constexpr int ST = 512;            // select: threads
constexpr int SW = ST / 32;
constexpr int BINS = 2048;
constexpr int KEYS = 24576;        // most keys held in shared memory (96 KB: two CTAs an SM; 16384 and below: three)
constexpr int MT = 256;            // move: threads that copy
constexpr int MR = 64;             // rows of a piece
constexpr int MC = 4;              // CTAs an SM

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
  unsigned* count;  // [B] pieces moved, and behind them the CTAs that are done
  unsigned* ready;  // [B] 1: to be moved
};

__device__ __forceinline__ bool evict_over(const EvictArgs& a, int L) { return L > a.limit && L <= a.g.capacity; }

// The bin that holds the `need`-th largest key (counted from the top bin), for all threads; need becomes its
// rank among that bin's keys.  The histogram is left at zero.
template <int BITS>
__device__ __forceinline__ int find_bin(unsigned* hist, int& need, int* s_scan, int* s_bin) {
  constexpr int PER = (1 << BITS) / ST;  // bins a thread, from the top
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  unsigned* first = hist + (1 << BITS) - (t + 1) * PER;  // (the thread's lowest bin)
  int c[PER], mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = first[PER - 1 - i];
    first[PER - 1 - i] = 0;
    mine += c[i];
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  const int of_warp = lane < SW ? s_scan[lane] : 0;
  int up = of_warp;  // the warps' sums, added up
#pragma unroll
  for (int o = 1; o < SW; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  int left = need - (__shfl_sync(0xffffffffu, up - of_warp, warp) + inc - mine);
  if (left > 0 && left <= mine) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (left > 0 && left <= c[i]) {
        s_bin[0] = (1 << BITS) - 1 - (t * PER + i);
        s_bin[1] = left;
      }
      left -= c[i];
    }
  }
  __syncthreads();
  need = s_bin[1];
  return s_bin[0];
}

__global__ void __launch_bounds__(ST, 3) evict_select_kernel(const EvictArgs a, const PagedEvictArgs p, int room) {
  extern __shared__ uint32_t keys[];
  __shared__ unsigned hist[BINS];
  __shared__ int s_scan[SW], s_bin[2], s_bad, s_gt[SW], s_eq[SW];
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int h = blockIdx.x % a.g.Hkv, bl = blockIdx.x / a.g.Hkv;
  const int l = bl % a.layers, b = bl / a.layers;
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
  int32_t* out = a.kept + ((static_cast<size_t>(l) * a.batch + b) * a.g.Hkv + h) * a.budget;
  for (int i = t; i < a.sink; i += ST) out[i] = i;
  for (int i = t; i < a.recent; i += ST) out[a.budget - a.recent + i] = L - a.recent + i;
  const int lo = a.sink, hi = L - a.recent;       // candidates: rows lo .. hi - 1
  int need = a.budget - a.sink - a.recent;        // of which these stay, fewer than there are (L > limit >= budget)
  if (need == 0) return;
  const float* w = p.w[l];
  const bool held = hi <= room;
  // four keys from row j (a multiple of 4, so of one page) on
  auto load_keys = [&](int j) {
    const float4 x = *reinterpret_cast<const float4*>(w + paged_row_or_zero(a.g, b, h, j, a.status));
    return make_uint4(weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w));
  };
  const int va = lo >> 2, vb = (hi + 3) >> 2;     // in fours; the first and the last may hold others' rows
  auto keys_of = [&](int v) { return held ? *reinterpret_cast<const uint4*>(keys + 4 * v) : load_keys(4 * v); };
  uint32_t prefix = 0;  // the threshold's bits so far
  for (int i = t; i < BINS; i += ST) hist[i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass == 2 ? 10 : 11, low = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    auto count = [&](uint4 k, int v) {
      const uint32_t x[4] = {k.x, k.y, k.z, k.w};
      const bool edge = v == va || v == vb - 1;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((pass == 0 || (x[e] >> (low + bits)) == (prefix >> (low + bits))) &&
            (!edge || (4 * v + e >= lo && 4 * v + e < hi)))
          atomicAdd(&hist[(x[e] >> low) & ((1u << bits) - 1)], 1u);
    };
    constexpr int U = 4;
    for (int v0 = va + t; v0 < vb; v0 += ST * U) {
      uint4 k[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + ST * u < vb) k[u] = pass == 0 ? load_keys(4 * (v0 + ST * u)) : keys_of(v0 + ST * u);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + ST * u;
        if (v >= vb) break;
        if (pass == 0 && held) *reinterpret_cast<uint4*>(keys + 4 * v) = k[u];
        count(k[u], v);
      }
    }
    __syncthreads();
    const int bin = pass == 2 ? find_bin<10>(hist, need, s_scan, s_bin) : find_bin<11>(hist, need, s_scan, s_bin);
    prefix |= static_cast<uint32_t>(bin) << low;
    __syncthreads();
  }
  // need: how many keys equal to the threshold stay (the lowest rows).  A warp takes a run of fours.
  const int per = (vb - va + SW - 1) / SW, w0 = min(vb, va + warp * per), w1 = min(vb, w0 + per);
  auto flags = [&](int v, unsigned& gt, unsigned& eq) {  // of four rows, a bit each
    const uint4 k = keys_of(v);
    gt = (k.x > prefix ? 1u : 0u) | (k.y > prefix ? 2u : 0u) | (k.z > prefix ? 4u : 0u) | (k.w > prefix ? 8u : 0u);
    eq = (k.x == prefix ? 1u : 0u) | (k.y == prefix ? 2u : 0u) | (k.z == prefix ? 4u : 0u) | (k.w == prefix ? 8u : 0u);
    unsigned in = 15u;
    if (v == va) in &= 15u << (lo & 3);
    if (v == vb - 1) in &= 15u >> (4 * vb - hi);
    gt &= in;
    eq &= in;
  };
  int gt = 0, eq = 0;
  for (int v = w0 + lane; v < w1; v += 32) {
    unsigned g, e;
    flags(v, g, e);
    gt += __popc(g);
    eq += __popc(e);
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
  for (int v0 = w0; v0 < w1; v0 += 32) {
    const int v = v0 + lane;
    unsigned g = 0, e = 0;
    if (v < w1) flags(v, g, e);
    const int mine = __popc(g) | (__popc(e) << 16);
    int inc = mine;  // (at most 128 each)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    int G = gt + ((inc - mine) & 0xffff), E = eq + ((inc - mine) >> 16);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if ((g >> x) & 1) {
        out[a.sink + G + min(E, need)] = 4 * v + x;
        ++G;
      } else if ((e >> x) & 1) {
        if (E < need) out[a.sink + G + E] = 4 * v + x;
        ++E;
      }
    }
    const int all = __shfl_sync(0xffffffffu, inc, 31);
    gt += all & 0xffff;
    eq += all >> 16;
  }
}

// Pieces of MR kept rows, in the order request (those to be moved), layer, head, piece.
__global__ void __launch_bounds__(MT + 32, MC) evict_move_kernel(const EvictArgs a, const PagedEvictArgs p, int chunks,
                                                            int vshift) {
  __shared__ int s_src[2][MR], s_dst[2][MR];
  __shared__ bool last;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int t = threadIdx.x, lane = t & 31;
  const int per_request = a.layers * a.g.Hkv * chunks;
  int live = 0;  // requests to be moved
  for (int b = 0; b < a.batch; b += 32)
    live += __popc(__ballot_sync(0xffffffffu, b + lane < a.batch && __ldcg(a.ready + b + lane) != 0));
  const long long total = static_cast<long long>(live) * per_request;
  const int u0 = static_cast<int>(total * blockIdx.x / gridDim.x), u1 = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  // the n-th request to be moved, by every warp for itself
  auto request = [&](int n) {
    for (int b = 0; b < a.batch; b += 32) {
      const unsigned m = __ballot_sync(0xffffffffu, b + lane < a.batch && __ldcg(a.ready + b + lane) != 0);
      if (n < __popc(m)) return b + static_cast<int>(__fns(m, 0, n + 1));
      n -= __popc(m);
    }
    return 0;  // (not met: there are `live` of them)
  };
  // a piece's rows (by the warp behind the others, two each), and their weights
  auto look_up = [&](int b, int v, int buf) {  // v: piece of the request
    const int group = v / chunks, n0 = (v - group * chunks) * MR;
    const int l = group / a.g.Hkv, h = group - l * a.g.Hkv;
    const int32_t* kept = a.kept + ((static_cast<size_t>(l) * a.batch + b) * a.g.Hkv + h) * a.budget;
    int r[2], page[2], src[2], dst[2];
    float w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int to = min(n0 + lane + 32 * e, a.budget - 1);
      r[e] = min(max(kept[to], 0), a.g.capacity - 1);
      page[e] = a.spare[static_cast<size_t>(b) * a.spare_pages + (to >> a.g.shift)];
      dst[e] = ((page[e] * a.g.Hkv + h) << a.g.shift) + (to & ((1 << a.g.shift) - 1));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) src[e] = paged_row_or_zero(a.g, b, h, r[e], a.status);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s_src[buf][lane + 32 * e] = src[e];
      s_dst[buf][lane + 32 * e] = dst[e];
      w[e] = p.w[l][src[e]];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (n0 + lane + 32 * e < a.budget) p.w[l][dst[e]] = w[e];
  };
  int n = u0 / per_request, v = u0 - n * per_request, b = 0, buf = 0, mine = 0;
  if (u0 < u1) {
    b = request(n);
    if (t >= MT) look_up(b, v, buf);
  }
  for (int u = u0; u < u1; ++u) {
    __syncthreads();  // (the piece's rows are there, and the other buffer's readers are done)
    const int group = v / chunks, rows = min(MR, a.budget - (v - group * chunks) * MR), l = group / a.g.Hkv, at_b = b;
    const bool over = v + 1 == per_request, ends = over || u + 1 == u1;
    v = over ? 0 : v + 1;
    if (over && u + 1 < u1) b = request(++n);
    if (t >= MT) {
      if (u + 1 < u1) look_up(b, v, buf ^ 1);
    } else {
      const uint4* k = static_cast<const uint4*>(p.k[l]);
      const uint4* vv = static_cast<const uint4*>(p.v[l]);
      uint4* kd = static_cast<uint4*>(p.k[l]);
      uint4* vd = static_cast<uint4*>(p.v[l]);
      const int vectors = rows << vshift, mask = (1 << vshift) - 1;
      constexpr int U = 2;  // a vector of K and one of V each
      for (int i0 = t; i0 < vectors; i0 += MT * U) {
        uint4 xk[U], xv[U];
#pragma unroll
        for (int x = 0; x < U; ++x) {
          const int i = i0 + x * MT;
          if (i < vectors) {
            const size_t at = (static_cast<size_t>(s_src[buf][i >> vshift]) << vshift) + (i & mask);
            xk[x] = __ldcs(k + at);
            xv[x] = __ldcs(vv + at);
          }
        }
#pragma unroll
        for (int x = 0; x < U; ++x) {
          const int i = i0 + x * MT;
          if (i < vectors) {
            const size_t at = (static_cast<size_t>(s_dst[buf][i >> vshift]) << vshift) + (i & mask);
            __stcs(kd + at, xk[x]);
            __stcs(vd + at, xv[x]);
          }
        }
      }
    }
    buf ^= 1;
    ++mine;
    if (!ends) continue;
    // this CTA's last piece of the request
    __threadfence();
    __syncthreads();
    if (t == 0) last = atomicAdd(&a.count[at_b], static_cast<unsigned>(mine)) == static_cast<unsigned>(per_request - mine);
    mine = 0;
    __syncthreads();
    if (!last) continue;
    __threadfence();
    for (int i = t; i < a.spare_pages; i += MT + 32) {
      int32_t* x = a.table + static_cast<size_t>(at_b) * a.g.max_pages + i;
      int32_t* y = a.spare + static_cast<size_t>(at_b) * a.spare_pages + i;
      const int32_t old = *x;
      *x = *y;
      *y = old;
    }
    if (t == 0) {
      a.seq_len[at_b] = a.budget;
      a.count[at_b] = 0;
    }
  }
  // the flags: by the last CTA of all, which have found their requests by them
  __syncthreads();
  if (t == 0) last = atomicAdd(a.count + a.batch, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  for (int i = t; i < a.batch; i += MT + 32) a.ready[i] = 0;
  if (t == 0) a.count[a.batch] = 0;
}

}  // namespace

size_t paged_evict_ws(const eagle_paged_evict_desc& d) { return (static_cast<size_t>(d.batch) * 8 + 4 + 15) / 16 * 16; }

cudaError_t launch_paged_evict(const eagle_paged_evict_desc& d, const PagedEvictArgs& p, int32_t* table,
                               int32_t* spare, int32_t* seq_len, int32_t* kept, uint32_t* status, void* ws,
                               int sms, cudaStream_t s) {
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
  a.ready = a.count + d.batch + 1;
  static unsigned long long configured = 0;
  cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(evict_select_kernel), KEYS * 4, configured);
  if (e != cudaSuccess) return e;
  const int groups = d.layers * d.batch * d.n_kv_heads, chunks = (d.budget + MR - 1) / MR;
  const int room = a.g.capacity < KEYS ? a.g.capacity : KEYS;  // (a multiple of 16)
  e = launch_pdl(evict_select_kernel, dim3(groups), dim3(ST), static_cast<size_t>(room) * 4, s, a, p, room);
  if (e != cudaSuccess) return e;
  const int bytes = d.head_dim * (d.dtype == EAGLE_F32 ? 4 : 2);
  const long long pieces = static_cast<long long>(groups) * chunks;
  const int ctas = static_cast<int>(pieces < sms * MC ? pieces : sms * MC);
  return launch_pdl(evict_move_kernel, dim3(ctas), dim3(MT + 32), 0, s, a, p, chunks,
                    bytes == 128 ? 3 : bytes == 256 ? 4 : 5);
}

}  // namespace eagle
