// kvq.cu -- the 8-bit KV cache: rows quantised as they are written, the accepted path
// appended to every layer's cache, rows read back.
//
// Same place in the step as kv_commit.cu (EAGLE review, section 3.3 and data path step 7:
// accepted tokens are appended; lesson "KV cache rollback"); the pages keep the cache in 16
// bits, the 8-bit form halves the bytes that tree attention streams.
//
// One thread group owns one 64-row block of one head, so a block's scale has one writer:
//   1. it loads the rows that fall into the block (all of them in flight at once, kept in
//      registers) and takes their largest magnitude;
//   2. the scale: that maximum's power of two, or the block's old scale if rows before the
//      first new one stay in the block and theirs is larger;
//   3. if the scale grew, the rows that stay are moved to it (their codes, not their
//      original values, which are gone);
//   4. the new rows' codes are stored.
// Each element is read once and written once; the write and read kernels are bound by HBM,
// the commit (a few rows per block) by the latency of its dependent loads.
#include "common.cuh"
#include "kvq.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace eagle {
namespace {

template <typename T>
struct Chunk;  // 8 consecutive elements of a row
template <>
struct Chunk<uint16_t> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

// Rows [lo, hi) of the block that begins at cache row `base`, by NT threads (tid in
// [0, NT), a multiple of 32; `red` NT / 32 floats; `bar` their named barrier): row r comes
// from src(r) (nullptr: the row is not written).  codes: the head's cache rows; scale: the
// block's entry.  D is a multiple of 8 and 64 * D / 8 chunks fit MAXC per thread.
template <typename T, int NT, int MAXC, typename Src>
__device__ __forceinline__ void put_block(int tid, float* red, int bar, int D, int base, int lo, int hi, Src src,
                                          uint8_t* codes, float* scale) {
  const int per = D / 8, total = (hi - lo) * per;
  Chunk<T> x[MAXC];
  bool on[MAXC];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    const int c = tid + i * NT;
    const T* p = c < total ? src(lo + c / per) : nullptr;
    on[i] = p != nullptr;
    if (on[i])
      x[i].load(p + (c % per) * 8);
    else
      x[i].zero();
  }
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    float f[8];
    x[i].get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = fabsf(f[e]);
      amax = fmaxf(amax, m <= 3.402823466e38f ? m : 0.f);  // the scale follows the finite values
    }
  }
  const bool holds = lo > base;  // rows before `lo` stay
  const float s_old = holds ? *scale : 0.f;
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  sm100::bar_sync(bar, NT);
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) amax = fmaxf(amax, red[w]);
  const float s = fmaxf(kvq_scale(amax), s_old);
  const float inv = kvq_inverse(s);
  if (s > s_old && s_old > 0.f) {
    const float ratio = s_old * inv;
    uint2* old = reinterpret_cast<uint2*>(codes + static_cast<size_t>(base) * D);
    for (int c = tid; c < (lo - base) * per; c += NT) {
      const uint2 w = old[c];
      old[c] = make_uint2(kvq_move4(w.x, ratio), kvq_move4(w.y, ratio));
    }
  }
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    if (!on[i]) continue;
    const int c = tid + i * NT;
    float f[8];
    x[i].get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    *reinterpret_cast<uint2*>(codes + static_cast<size_t>(lo) * D + static_cast<size_t>(c) * 8) =
        make_uint2(kvq_code2(f[0], f[1]) | (kvq_code2(f[2], f[3]) << 16),
                   kvq_code2(f[4], f[5]) | (kvq_code2(f[6], f[7]) << 16));
  }
  sm100::bar_sync(bar, NT);  // every thread has read the old scale and `red`
  if (tid == 0) *scale = s;
}

// A request's row span: valid if it lies inside the cache.
__device__ __forceinline__ bool span(const eagle_kvq_desc& d, const int32_t* start, const int32_t* count, int b,
                                     int& first, int& n) {
  first = start[b];
  n = count ? count[b] : d.rows;
  return first >= 0 && n >= 0 && n <= d.rows && first <= d.max_seq - n;
}

// grid (blocks a span can touch, B Hkv, K / V) x 256
template <typename T>
__global__ void __launch_bounds__(256) kvq_write_kernel(const eagle_kvq_desc d, const T* k, const T* v,
                                                        const int32_t* start, const int32_t* count, uint8_t* k8,
                                                        float* ks, uint8_t* v8, float* vs, uint32_t* status) {
  __shared__ float red[8];
  const int bh = blockIdx.y, b = bh / d.n_kv_heads;
  int first, n;
  if (!span(d, start, count, b, first, n)) {
    if (status && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, EAGLE_STATUS_CACHE_FULL);
    return;
  }
  const int blk = first / kQB + blockIdx.x;
  const int base = blk * kQB;
  const int lo = max(first, base), hi = min(first + n, base + kQB);
  if (lo >= hi) return;
  const T* x = (blockIdx.z ? v : k) + static_cast<size_t>(bh) * d.rows * d.head_dim;
  const int nblk = (d.max_seq + kQB - 1) / kQB;
  put_block<T, 256, 4>(
      threadIdx.x, red, 1, d.head_dim, base, lo, hi,
      [&](int r) { return x + static_cast<size_t>(r - first) * d.head_dim; },
      (blockIdx.z ? v8 : k8) + static_cast<size_t>(bh) * d.max_seq * d.head_dim,
      (blockIdx.z ? vs : ks) + static_cast<size_t>(bh) * nblk + blk);
}

// Read back: a thread takes 16 output bytes at a time (8 bf16 or 4 fp32 elements), four of
// them in flight.  grid (chunks, B Hkv, K / V) x 256
template <bool F32>
__global__ void __launch_bounds__(256) kvq_read_kernel(const eagle_kvq_desc d, const uint8_t* k8, const float* ks,
                                                       const uint8_t* v8, const float* vs, const int32_t* start,
                                                       const int32_t* count, void* k, void* v, uint32_t* status) {
  constexpr int E = F32 ? 4 : 8, U = 4;
  const int bh = blockIdx.y, b = bh / d.n_kv_heads, D = d.head_dim;
  int first, n;
  if (!span(d, start, count, b, first, n)) {
    if (status && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, EAGLE_STATUS_CACHE_FULL);
    return;
  }
  const int per = D / E;
  const long long total = static_cast<long long>(n) * per;
  const int nblk = (d.max_seq + kQB - 1) / kQB;
  const uint8_t* src = (blockIdx.z ? v8 : k8) + (static_cast<size_t>(bh) * d.max_seq + first) * D;
  const float* sc = (blockIdx.z ? vs : ks) + static_cast<size_t>(bh) * nblk;
  uint8_t* dst = static_cast<uint8_t*>(blockIdx.z ? v : k) + static_cast<size_t>(bh) * d.rows * D * (F32 ? 4 : 2);
  const long long c0 = static_cast<long long>(blockIdx.x) * (256 * U) + threadIdx.x;
  uint2 w[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long c = c0 + u * 256;
    if (c >= total) continue;
    if (F32)
      w[u].x = __ldg(reinterpret_cast<const uint32_t*>(src) + c);
    else
      w[u] = __ldg(reinterpret_cast<const uint2*>(src) + c);
    s[u] = __ldg(sc + (first + static_cast<int>(c / per)) / kQB);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long c = c0 + u * 256;
    if (c >= total) continue;
    const float2 a = kvq_float2(w[u].x), e = kvq_float2(w[u].x >> 16);
    // a scale of 0 marks a block of zeros, whatever its codes
    const float z = s[u];
    auto val = [&](float code) { return z > 0.f ? code * z : 0.f; };
    if (F32) {
      reinterpret_cast<float4*>(dst)[c] = make_float4(val(a.x), val(a.y), val(e.x), val(e.y));
    } else {
      const float2 f = kvq_float2(w[u].y), g = kvq_float2(w[u].y >> 16);
      auto two = [&](float2 t) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(val(t.x), val(t.y));
        return *reinterpret_cast<const uint32_t*>(&r);
      };
      reinterpret_cast<uint4*>(dst)[c] = make_uint4(two(a), two(e), two(f), two(g));
    }
  }
}

// grid (Hkv, B, layers) x 256: threads 0..127 take K, 128..255 V of one head.
template <typename T>
__global__ void __launch_bounds__(256) kvq_commit_kernel(const eagle_commit_desc d,
                                                         const __grid_constant__ KvqCommitArgs a,
                                                         const int32_t* n_acc, const int32_t* path,
                                                         const int32_t* seq_len, void* feat_cache,
                                                         const void* tree_feat) {
  __shared__ float red[8];
  __shared__ int node[kMaxRows];
  const int h = blockIdx.x, b = blockIdx.y, l = blockIdx.z;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  if (!commit_fits(d, n_acc, seq_len, b)) return;
  const int first = seq_len[b], n = n_acc[b] + 1;
  for (int m = threadIdx.x; m < n; m += 256) {
    const int r = path[static_cast<size_t>(b) * (d.max_depth + 1) + m];
    node[m] = r >= 0 && r < d.rows ? r : -1;  // a bad node is flagged by the finalize kernel, its row left as it was
  }
  __syncthreads();
  const int half = threadIdx.x >> 7, tid = threadIdx.x & 127, D = d.head_dim;
  const size_t bh = static_cast<size_t>(b) * d.n_kv_heads + h;
  const int nblk = (d.max_seq + kQB - 1) / kQB;
  const T* tree = static_cast<const T*>(half ? a.tree_v[l] : a.tree_k[l]) + bh * d.rows * D;
  uint8_t* codes = static_cast<uint8_t*>(half ? a.v8[l] : a.k8[l]) + bh * d.max_seq * D;
  float* scale = (half ? a.vs[l] : a.ks[l]) + bh * nblk;
  for (int blk = first / kQB; blk * kQB < first + n; ++blk) {
    const int base = blk * kQB;
    put_block<T, 128, 8>(
        tid, red + 4 * half, 1 + half, D, base, max(first, base), min(first + n, base + kQB),
        [&](int r) -> const T* {
          const int nd = node[r - first];
          return nd < 0 ? nullptr : tree + static_cast<size_t>(nd) * D;
        },
        codes, scale + blk);
  }
  if (h == 0 && l == 0 && d.feat_dim > 0) {
    const size_t bytes = static_cast<size_t>(d.feat_dim) * (d.feat_dtype == EAGLE_F32 ? 4 : 2);
    for (int m = 0; m < n; ++m) {
      if (node[m] < 0) continue;
      const uint8_t* s = static_cast<const uint8_t*>(tree_feat) + (static_cast<size_t>(b) * d.rows + node[m]) * bytes;
      uint8_t* t = static_cast<uint8_t*>(feat_cache) + (static_cast<size_t>(b) * d.max_seq + first + m) * bytes;
      if (bytes % 16 == 0)
        for (size_t i = threadIdx.x; i < bytes / 16; i += 256)
          reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(s)[i];
      else
        for (size_t i = threadIdx.x; i < bytes; i += 256) t[i] = s[i];
    }
  }
}

// A plain launch when pdl is false; a programmatic one (the kernel's griddepcontrol.wait
// orders it after the preceding kernel) otherwise.
template <typename... P, typename... A>
cudaError_t launch(void (*k)(P...), dim3 grid, int threads, cudaStream_t s, bool pdl, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kvq_write(const eagle_kvq_desc& d, const void* k, const void* v, const int32_t* start,
                             const int32_t* count, uint8_t* k8, float* ks, uint8_t* v8, float* vs, uint32_t* status,
                             cudaStream_t s) {
  const dim3 grid((d.rows + 2 * kQB - 2) / kQB, d.batch * d.n_kv_heads, 2);
  if (d.dtype == EAGLE_F32)
    return launch(kvq_write_kernel<float>, grid, 256, s, false, d, static_cast<const float*>(k),
                  static_cast<const float*>(v), start, count, k8, ks, v8, vs, status);
  return launch(kvq_write_kernel<uint16_t>, grid, 256, s, false, d, static_cast<const uint16_t*>(k),
                static_cast<const uint16_t*>(v), start, count, k8, ks, v8, vs, status);
}

cudaError_t launch_kvq_read(const eagle_kvq_desc& d, const uint8_t* k8, const float* ks, const uint8_t* v8,
                            const float* vs, const int32_t* start, const int32_t* count, void* k, void* v,
                            uint32_t* status, cudaStream_t s) {
  const bool f32 = d.dtype == EAGLE_F32;
  const long long chunks = static_cast<long long>(d.rows) * d.head_dim / (f32 ? 4 : 8);
  const dim3 grid(static_cast<unsigned>((chunks + 1023) / 1024), d.batch * d.n_kv_heads, 2);
  return f32 ? launch(kvq_read_kernel<true>, grid, 256, s, false, d, k8, ks, v8, vs, start, count, k, v, status)
             : launch(kvq_read_kernel<false>, grid, 256, s, false, d, k8, ks, v8, vs, start, count, k, v, status);
}

cudaError_t launch_kvq_commit(const eagle_commit_desc& d, const KvqCommitArgs& a, const int32_t* n_acc,
                              const int32_t* path, int32_t* seq_len, int32_t* commit_pos, void* feat_cache,
                              const void* tree_feat, uint32_t* status, cudaStream_t s) {
  const dim3 grid(d.n_kv_heads, d.batch, d.layers);
  const int32_t* len = seq_len;
  cudaError_t e = d.dtype == EAGLE_F32
                      ? launch(kvq_commit_kernel<float>, grid, 256, s, true, d, a, n_acc, path, len, feat_cache, tree_feat)
                      : launch(kvq_commit_kernel<uint16_t>, grid, 256, s, true, d, a, n_acc, path, len, feat_cache,
                               tree_feat);
  if (e != cudaSuccess) return e;
  return launch_commit_finalize(d, n_acc, path, seq_len, commit_pos, status, s);
}

}  // namespace eagle
