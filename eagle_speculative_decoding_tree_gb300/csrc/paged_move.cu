// paged_move.cu -- K/V rows into a paged cache: prompts and new tokens (eagle_paged_write), and the
// accepted path of every layer (eagle_paged_commit).  Copies of whole rows, 16 bytes a thread and load;
// bound by memory for prompts and by the launch for a few rows.
#include "paged.cuh"

namespace eagle {
namespace {

constexpr int WT = 256;  // threads
constexpr int WV = 4;    // 16-byte vectors a thread moves of K, and of V, all loads in flight together

// One CTA: WT * WV vectors of one request's rows, taken as [Hkv * N] rows in memory order (so that the
// heads of a single new token share a CTA).  vshift: log2 of the 16-byte vectors of a row.
__global__ void __launch_bounds__(WT) paged_write_kernel(const PagedGeom g, int N, int vshift, const uint4* k,
                                                         const uint4* v, const int32_t* start, const int32_t* count,
                                                         uint4* kp, uint4* vp, uint32_t* status) {
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int b = blockIdx.y;
  const int first = start[b], n = count ? count[b] : N;
  if (n < 0 || n > N || first < 0 || first > g.capacity - n) {
    if (status && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, EAGLE_STATUS_CACHE_FULL);
    return;
  }
  const long long total = (static_cast<long long>(g.Hkv) * N) << vshift;
  const size_t src0 = static_cast<size_t>(b) * total;
  uint4 xk[WV], xv[WV];
  long long to[WV];
#pragma unroll
  for (int i = 0; i < WV; ++i) {
    const long long at = static_cast<long long>(blockIdx.x) * (WT * WV) + i * WT + threadIdx.x;
    to[i] = -1;
    if (at < total) {
      const unsigned row = static_cast<unsigned>(at >> vshift);  // h * N + r
      const unsigned h = row / static_cast<unsigned>(N), r = row - h * N;
      if (static_cast<int>(r) < n) {
        xk[i] = k[src0 + at];
        xv[i] = v[src0 + at];
        const int y = paged_row(g, b, h, first + r);
        to[i] = y < 0 ? -2 : (static_cast<long long>(y) << vshift) + (at & ((1 << vshift) - 1));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < WV; ++i) {
    if (to[i] >= 0) {
      kp[to[i]] = xk[i];
      vp[to[i]] = xv[i];
    } else if (to[i] == -2 && status) {
      atomicOr(status, EAGLE_STATUS_BAD_PAGE);
    }
  }
}

constexpr int CT = 256;  // threads: a 16-byte vector of K and one of V each, of every layer

__device__ __forceinline__ bool paged_commit_fits(const eagle_paged_commit_desc& d, int capacity, int na, int L) {
  return na >= 0 && na <= d.max_depth && L >= 0 && L <= capacity - 1 - na;
}

constexpr int CL = 4;    // layers a CTA takes: 8 loads a thread in flight

// grid (vectors of a request's path rows / CT, B, L / CL).  Every CTA reads the old length; the last one of its
// request to finish (counters in ws) writes the new one, so that one launch does.
__global__ void __launch_bounds__(CT) paged_commit_kernel(const eagle_paged_commit_desc d, const PagedGeom g,
                                                          const CommitArgs a, int vshift, const int32_t* n_acc,
                                                          const int32_t* path, int32_t* seq_len, int32_t* commit_pos,
                                                          uint8_t* feat_pages, const uint8_t* tree_feat,
                                                          uint32_t* status, unsigned* counter) {
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int b = blockIdx.y, l0 = blockIdx.z * CL, maxp = d.max_depth + 1;
  const int na = n_acc[b], L = seq_len[b];
  const bool fits = paged_commit_fits(d, g.capacity, na, L);
  if (fits) {
    // vectors in the order path row, head, vector
    const int at = blockIdx.x * CT + threadIdx.x;
    const int c = at & ((1 << vshift) - 1), row = at >> vshift;
    const int m = row / g.Hkv, h = row - m * g.Hkv;
    if (m <= na) {
      const int node = path[static_cast<size_t>(b) * maxp + m];
      const int y = paged_row(g, b, h, L + m);
      if (node >= 0 && node < d.rows && y >= 0) {
        const size_t src = (((static_cast<size_t>(b) * g.Hkv + h) * d.rows + node) << vshift) + c;
        const size_t dst = (static_cast<size_t>(y) << vshift) + c;
        uint4 xk[CL], xv[CL];
#pragma unroll
        for (int i = 0; i < CL; ++i)
          if (l0 + i < d.layers) {
            xk[i] = static_cast<const uint4*>(a.tree_k[l0 + i])[src];
            xv[i] = static_cast<const uint4*>(a.tree_v[l0 + i])[src];
          }
#pragma unroll
        for (int i = 0; i < CL; ++i)
          if (l0 + i < d.layers) {
            static_cast<uint4*>(a.k_cache[l0 + i])[dst] = xk[i];
            static_cast<uint4*>(a.v_cache[l0 + i])[dst] = xv[i];
          }
      }
    }
    if (l0 == 0 && d.feat_dim > 0 && blockIdx.x == 0) {
      const size_t bytes = static_cast<size_t>(d.feat_dim) * (d.feat_dtype == EAGLE_F32 ? 4 : 2);
      for (int i = 0; i <= na; ++i) {
        const int node = path[static_cast<size_t>(b) * maxp + i];
        const int r = L + i;
        const int page = g.table[static_cast<size_t>(b) * g.max_pages + (r >> g.shift)];
        if (node < 0 || node >= d.rows || static_cast<unsigned>(page) >= static_cast<unsigned>(g.n_pages)) continue;
        const uint8_t* src = tree_feat + (static_cast<size_t>(b) * d.rows + node) * bytes;
        uint8_t* dst =
            feat_pages + ((static_cast<size_t>(page) << g.shift) + (r & ((1 << g.shift) - 1))) * bytes;
        if (bytes % 16 == 0) {
          for (size_t j = threadIdx.x; j < bytes / 16; j += CT)
            reinterpret_cast<uint4*>(dst)[j] = reinterpret_cast<const uint4*>(src)[j];
        } else {
          for (size_t j = threadIdx.x; j < bytes / 2; j += CT)
            reinterpret_cast<uint16_t*>(dst)[j] = reinterpret_cast<const uint16_t*>(src)[j];
        }
      }
    }
  }
  __shared__ bool last;
  __syncthreads();  // (everyone has the old length)
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(counter + b, 1u) == gridDim.x * gridDim.z - 1;
    if (last) counter[b] = 0;
  }
  __syncthreads();
  if (!last) return;
  uint32_t st = fits ? 0 : EAGLE_STATUS_CACHE_FULL;
  for (int m = threadIdx.x; m < maxp; m += CT) {
    const bool on = fits && m <= na;
    if (on) {
      const int node = path[static_cast<size_t>(b) * maxp + m];
      if (node < 0 || node >= d.rows) st |= EAGLE_STATUS_BAD_TREE;
      if (paged_row(g, b, 0, L + m) < 0) st |= EAGLE_STATUS_BAD_PAGE;
    }
    if (commit_pos) commit_pos[static_cast<size_t>(b) * maxp + m] = on ? L + m : -1;
  }
  if (fits && threadIdx.x == 0) seq_len[b] = L + na + 1;
  if (st && status) atomicOr(status, st);
}

int vector_shift(int head_dim, int dtype) {  // 16-byte vectors of a row: 8, 16 or 32
  const int bytes = head_dim * (dtype == EAGLE_F32 ? 4 : 2);
  return bytes == 128 ? 3 : bytes == 256 ? 4 : 5;
}

}  // namespace

cudaError_t launch_paged_write(const eagle_paged_desc& d, const void* k, const void* v, const int32_t* table,
                               const int32_t* start, const int32_t* count, void* k_pages, void* v_pages,
                               uint32_t* status, cudaStream_t s) {
  const PagedGeom g = paged_geom(table, d.n_pages, d.max_pages, d.page_size, d.n_kv_heads);
  const int vshift = vector_shift(d.head_dim, d.dtype);
  const long long total = (static_cast<long long>(d.n_kv_heads) * d.rows) << vshift;
  const dim3 grid(static_cast<unsigned>((total + WT * WV - 1) / (WT * WV)), d.batch);
  return launch_pdl(paged_write_kernel, grid, dim3(WT), 0, s, g, d.rows, vshift, static_cast<const uint4*>(k),
                    static_cast<const uint4*>(v), start, count, static_cast<uint4*>(k_pages),
                    static_cast<uint4*>(v_pages), status);
}

size_t paged_commit_ws(const eagle_paged_commit_desc& d) { return (static_cast<size_t>(d.batch) * 4 + 15) / 16 * 16; }

cudaError_t launch_paged_commit(const eagle_paged_commit_desc& d, const CommitArgs& a, const int32_t* table,
                                const int32_t* n_acc, const int32_t* path, int32_t* seq_len, int32_t* commit_pos,
                                void* feat_pages, const void* tree_feat, uint32_t* status, void* ws, cudaStream_t s) {
  const PagedGeom g = paged_geom(table, d.n_pages, d.max_pages, d.page_size, d.n_kv_heads);
  const int vshift = vector_shift(d.head_dim, d.dtype);
  const int vectors = ((d.max_depth + 1) * d.n_kv_heads) << vshift;
  const dim3 grid((vectors + CT - 1) / CT, d.batch, (d.layers + CL - 1) / CL);
  return launch_pdl(paged_commit_kernel, grid, dim3(CT), 0, s, d, g, a, vshift, n_acc, path, seq_len, commit_pos,
                    static_cast<uint8_t*>(feat_pages), static_cast<const uint8_t*>(tree_feat), status,
                    static_cast<unsigned*>(ws));
}

}  // namespace eagle
