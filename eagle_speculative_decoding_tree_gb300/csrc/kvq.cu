// kvq.cu -- the 8-bit KV cache: rows quantised as they are written, the accepted path
// appended to every layer's cache, rows read back.
//
// Same place in the step as kv_commit.cu (EAGLE review, section 3.3 and data path step 7:
// accepted tokens are appended; lesson "KV cache rollback"); the pages keep the cache in 16
// bits, the 8-bit form halves the bytes that tree attention streams.
//
// One owner per 64-row block of one head (a CTA when writing, a warp when committing), so a
// block's scale has one writer:
//   1. it loads the rows that fall into the block (kept in registers) and takes their largest
//      magnitude;
//   2. the scale: that maximum's power of two, or the block's old scale if rows before the
//      first new one stay in the block and theirs is larger;
//   3. if the scale grew, the rows that stay are moved to it (their codes, not their
//      original values, which are gone);
//   4. the new rows' codes are stored.
// Each element is read once and written once.  Writing and reading are bound by HBM: the write
// kernel's CTAs are persistent and hold the next block's rows in flight while they finish one
// (one block at a time leaves HBM idle through every block's reduction).  A commit is a few rows
// for each of layers x requests x heads blocks, bound by the latency of its dependent loads
// (lengths, path, rows), so it takes a warp per block and all of them at once.
// Measured (8 heads x 128, bf16): 8192 rows written in 7.9 us from L2, 12.5 from HBM (50 MB; a CTA per
// block, one block at a time, took 15.5 from L2), 32 requests of 511 to 1021 rows 31.9 us, 8192 rows
// read back in 6.3; 32 layers' accepted path of one request committed in 5.3 us, of 32 requests in
// 11.8 (74 by a CTA per block).
#include <algorithm>

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

// The largest magnitude of a chunk as float bits (ordered as integers; NaN and infinities are at
// or above kInf).  On the bits, two bf16 elements an instruction: the float way, with its test of
// every element, took as many issue slots as the loads and stores together.
constexpr uint32_t kInf = 0x7f800000u;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t chunk_max(const Chunk<uint16_t>& x) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t r = max_u16x2(max_u16x2(x.u.x & m, x.u.y & m), max_u16x2(x.u.z & m, x.u.w & m));
  return max(r << 16, r & 0xffff0000u);
}
__device__ __forceinline__ uint32_t chunk_max(const Chunk<float>& x) {
  float f[8];
  x.get(f);
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) r = max(r, __float_as_uint(f[e]) & 0x7fffffffu);
  return r;
}
// ... of its finite values: what the scale follows in a block that has others.
template <typename T>
__device__ __forceinline__ uint32_t chunk_finite_max(const Chunk<T>& x) {
  float f[8];
  x.get(f);
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(f[e]) & 0x7fffffffu;
    r = b < kInf ? max(r, b) : r;
  }
  return r;
}

__device__ __forceinline__ uint32_t code2_of_finite(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// special: the block has values that are not finite.
template <typename T>
__device__ __forceinline__ uint2 chunk_codes(const Chunk<T>& x, float inv, bool special) {
  float f[8];
  x.get(f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= inv;
  if (special)
    return make_uint2(kvq_code2(f[0], f[1]) | (kvq_code2(f[2], f[3]) << 16),
                      kvq_code2(f[4], f[5]) | (kvq_code2(f[6], f[7]) << 16));
  return make_uint2(code2_of_finite(f[0], f[1]) | (code2_of_finite(f[2], f[3]) << 16),
                    code2_of_finite(f[4], f[5]) | (code2_of_finite(f[6], f[7]) << 16));
}

// The rows [base, lo) that stay in a block whose scale grew, ratio = old scale / new (0 for rows
// under a scale of 0: whatever their finite codes, they are zeros), by threads tid of n.
__device__ __forceinline__ void move_rows(uint8_t* codes, int D, int base, int lo, float ratio, int tid, int n) {
  uint2* old = reinterpret_cast<uint2*>(codes + static_cast<size_t>(base) * D);
  for (int c = tid; c < (lo - base) * (D / 8); c += n) {
    const uint2 w = old[c];
    old[c] = make_uint2(kvq_move4(w.x, ratio), kvq_move4(w.y, ratio));
  }
}

// A request's row span: valid if it lies inside the cache.
__device__ __forceinline__ bool span(const eagle_kvq_desc& d, const int32_t* start, const int32_t* count, int b,
                                     int& first, int& n) {
  first = start[b];
  n = count ? count[b] : d.rows;
  return first >= 0 && n >= 0 && n <= d.rows && first <= d.max_seq - n;
}

constexpr int kWriteThreads = 128;

// One block of the write kernel's work list (which: K or V; block of the request's span).
template <typename T>
struct WriteItem {
  static constexpr int C = 64 * 128 / 8 / kWriteThreads;  // chunks of a thread
  Chunk<T> x[C];
  uint8_t* codes;  // the head's rows
  float* scale;
  int base, lo, hi;  // empty: lo >= hi

  __device__ __forceinline__ void fetch(const eagle_kvq_desc& d, int item, int per_head, int items, const T* k, const T* v,
                                        const int32_t* start, const int32_t* count, uint8_t* k8, float* ks,
                                        uint8_t* v8, float* vs, uint32_t* status) {
    lo = hi = 0;
    if (item >= items) return;
    const int j = item % per_head, hv = item / per_head;
    const int which = hv & 1, bh = hv >> 1, b = bh / d.n_kv_heads;
    int first, n;
    if (!span(d, start, count, b, first, n)) {
      if (status && j == 0 && threadIdx.x == 0) atomicOr(status, EAGLE_STATUS_CACHE_FULL);
      return;
    }
    const int blk = first / kQB + j;
    base = blk * kQB;
    lo = max(first, base);
    hi = min(first + n, base + kQB);
    if (lo >= hi) return;
    const T* src = (which ? v : k) + (static_cast<size_t>(bh) * d.rows + (lo - first)) * d.head_dim;
    const int total = (hi - lo) * (d.head_dim / 8);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = threadIdx.x + i * kWriteThreads;
      if (c < total)
        x[i].load(src + static_cast<size_t>(c) * 8);
      else
        x[i].zero();
    }
    codes = (which ? v8 : k8) + static_cast<size_t>(bh) * d.max_seq * d.head_dim;
    scale = (which ? vs : ks) + static_cast<size_t>(bh) * ((d.max_seq + kQB - 1) / kQB) + blk;
  }
};

// Persistent: CTA c takes the blocks c, c + grid, ... of the list
template <typename T>
__global__ void __launch_bounds__(kWriteThreads) kvq_write_kernel(const eagle_kvq_desc d, int per_head, int items, const T* k,
                                                        const T* v, const int32_t* start, const int32_t* count,
                                                        uint8_t* k8, float* ks, uint8_t* v8, float* vs,
                                                        uint32_t* status) {
  __shared__ uint32_t red[2][kWriteThreads / 32];
  WriteItem<T> cur, nxt;
  cur.fetch(d, blockIdx.x, per_head, items, k, v, start, count, k8, ks, v8, vs, status);
  int turn = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    nxt.fetch(d, item + gridDim.x, per_head, items, k, v, start, count, k8, ks, v8, vs, status);
    if (cur.lo < cur.hi) {  // the same for the whole CTA
      const float s_old = cur.lo > cur.base ? *cur.scale : 0.f;
      auto reduce = [&](uint32_t m) {  // over the CTA; the halves of `red` take turns
        m = __reduce_max_sync(0xffffffffu, m);
        if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWriteThreads / 32; ++w) m = max(m, red[turn][w]);
        turn ^= 1;
        return m;
      };
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < cur.C; ++i) m = max(m, chunk_max(cur.x[i]));
      m = reduce(m);
      const bool special = m >= kInf;
      if (special) {
        m = 0;
#pragma unroll
        for (int i = 0; i < cur.C; ++i) m = max(m, chunk_finite_max(cur.x[i]));
        m = reduce(m);
      }
      const float s = fmaxf(kvq_scale(__uint_as_float(m)), s_old), inv = kvq_inverse(s);
      if (s > s_old && cur.lo > cur.base) move_rows(cur.codes, d.head_dim, cur.base, cur.lo, s_old * inv, threadIdx.x, kWriteThreads);
      const int total = (cur.hi - cur.lo) * (d.head_dim / 8);
      uint2* dst = reinterpret_cast<uint2*>(cur.codes + static_cast<size_t>(cur.lo) * d.head_dim);
#pragma unroll
      for (int i = 0; i < cur.C; ++i) {
        const int c = threadIdx.x + i * kWriteThreads;
        if (c < total) dst[c] = chunk_codes(cur.x[i], inv, special);
      }
      if (threadIdx.x == 0) *cur.scale = s;
    }
    cur = nxt;
  }
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
  const int lg = 31 - __clz(D / E);  // a row's pieces: a power of two (64-bit divisions cost more than all else here)
  const long long total = static_cast<long long>(n) << lg;
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
    s[u] = __ldg(sc + (first + static_cast<int>(c >> lg)) / kQB);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long c = c0 + u * 256;
    if (c >= total) continue;
    const float2 a = kvq_float2(w[u].x), e = kvq_float2(w[u].x >> 16);
    const float z = s[u];
    auto val = [&](float code) { return code * z; };  // (a NaN code under any scale, 0 too, is NaN)
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

// A warp per (layer, request, KV head): the path's rows of K and V into the one or two blocks
// they fall in.  16 bytes (bf16) of a row per lane: two rows of 128 at a time, four such loads of
// K and of V in flight; paths longer than that take further rounds, read twice.
template <typename T>
__global__ void __launch_bounds__(128) kvq_commit_kernel(const eagle_commit_desc d,
                                                         const __grid_constant__ KvqCommitArgs a,
                                                         const int32_t* n_acc, const int32_t* path,
                                                         const int32_t* seq_len, void* feat_cache,
                                                         const void* tree_feat) {
  constexpr int C = 4;
  const int lane = threadIdx.x & 31;
  const int id = blockIdx.x * 4 + (threadIdx.x >> 5), per = d.n_kv_heads * d.batch;  // (layers <= 128, per <= 65535)
  const int l = id / per, bh = id % per, b = bh / d.n_kv_heads, h = bh % d.n_kv_heads;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  if (l >= d.layers || !commit_fits(d, n_acc, seq_len, b)) return;
  const int first = seq_len[b], n = n_acc[b] + 1, D = d.head_dim;
  const int32_t* nodes = path + static_cast<size_t>(b) * (d.max_depth + 1);
  const int lanes = D / 8, rpp = 32 / lanes, sub = lane / lanes, col = (lane % lanes) * 8;
  const int nblk = (d.max_seq + kQB - 1) / kQB;
  const size_t hb = static_cast<size_t>(bh);
  for (int blk = first / kQB; blk * kQB < first + n; ++blk) {
    const int base = blk * kQB, lo = max(first, base), hi = min(first + n, base + kQB);
    const T* tree[2] = {static_cast<const T*>(a.tree_k[l]) + hb * d.rows * D + col,
                        static_cast<const T*>(a.tree_v[l]) + hb * d.rows * D + col};
    uint8_t* codes[2] = {static_cast<uint8_t*>(a.k8[l]) + hb * d.max_seq * D,
                         static_cast<uint8_t*>(a.v8[l]) + hb * d.max_seq * D};
    float* scale[2] = {a.ks[l] + hb * nblk + blk, a.vs[l] + hb * nblk + blk};
    // rows lo + r0 + sub + rpp i; a bad node (flagged by the finalize kernel) writes nothing
    Chunk<T> x[2][C];
    int row[C];
    auto fetch = [&](int r0) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int r = lo + r0 + sub + rpp * i;
        row[i] = -1;
        if (r < hi) {
          const int nd = __ldg(nodes + (r - first));
          if (nd >= 0 && nd < d.rows) row[i] = nd;
        }
      }
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < C; ++i) {
          if (row[i] >= 0)
            x[w][i].load(tree[w] + static_cast<size_t>(row[i]) * D);
          else
            x[w][i].zero();
        }
    };
    fetch(0);
    float s_old[2] = {0.f, 0.f}, s[2];
    uint32_t m[2] = {0u, 0u};
    if (lo > base) {
      s_old[0] = *scale[0];
      s_old[1] = *scale[1];
    }
    const int round = C * rpp, rounds = (hi - lo + round - 1) / round;
    for (int g = 0; g < rounds; ++g) {
      if (g > 0) fetch(g * round);
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < C; ++i) m[w] = max(m[w], chunk_max(x[w][i]));
    }
    bool special[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      m[w] = __reduce_max_sync(0xffffffffu, m[w]);
      special[w] = m[w] >= kInf;
    }
    if (special[0] || special[1]) {
      uint32_t fin[2] = {0u, 0u};
      for (int g = 0; g < rounds; ++g) {  // (again, ending with the last round's rows)
        fetch(g * round);
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < C; ++i) fin[w] = max(fin[w], chunk_finite_max(x[w][i]));
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) m[w] = __reduce_max_sync(0xffffffffu, fin[w]);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      s[w] = fmaxf(kvq_scale(__uint_as_float(m[w])), s_old[w]);
      if (s[w] > s_old[w] && lo > base) move_rows(codes[w], D, base, lo, s_old[w] * kvq_inverse(s[w]), lane, 32);
    }
    for (int g = rounds - 1; g >= 0; --g) {  // (the last round's rows are still in registers)
      if (g < rounds - 1) fetch(g * round);
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (row[i] >= 0)
            *reinterpret_cast<uint2*>(codes[w] + static_cast<size_t>(lo + g * round + sub + rpp * i) * D + col) =
                chunk_codes(x[w][i], kvq_inverse(s[w]), special[w]);
    }
    __syncwarp();  // every lane has read the old scales
    if (lane < 2) *(lane ? scale[1] : scale[0]) = lane ? s[1] : s[0];
  }
  if (d.feat_dim > 0) {
    // feature rows in pieces of 2 KB, shared out over the request's warps
    const size_t bytes = static_cast<size_t>(d.feat_dim) * (d.feat_dtype == EAGLE_F32 ? 4 : 2);
    const int pieces = static_cast<int>((bytes + 2047) / 2048);
    for (int u = l * d.n_kv_heads + h; u < n * pieces; u += d.layers * d.n_kv_heads) {
      const int m = u / pieces, nd = nodes[m];
      if (nd < 0 || nd >= d.rows) continue;
      const size_t off = static_cast<size_t>(u % pieces) * 2048, end = off + 2048 < bytes ? off + 2048 : bytes;
      const uint8_t* src = static_cast<const uint8_t*>(tree_feat) + (static_cast<size_t>(b) * d.rows + nd) * bytes;
      uint8_t* dst = static_cast<uint8_t*>(feat_cache) + (static_cast<size_t>(b) * d.max_seq + first + m) * bytes;
      if (bytes % 16 == 0) {
#pragma unroll 4
        for (size_t i = off + lane * 16; i < end; i += 512)
          *reinterpret_cast<uint4*>(dst + i) = __ldg(reinterpret_cast<const uint4*>(src + i));
      } else {
        for (size_t i = off + lane; i < end; i += 32) dst[i] = src[i];
      }
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
                             int num_sms, cudaStream_t s) {
  const int per_head = static_cast<int>(kvq_span_blocks(d.rows));
  const long long items = 2ll * per_head * d.batch * d.n_kv_heads;
  const int grid = static_cast<int>(std::min<long long>(items, (d.dtype == EAGLE_F32 ? 3ll : 4ll) * num_sms));  // CTAs that fit
  if (d.dtype == EAGLE_F32)
    return launch(kvq_write_kernel<float>, dim3(grid), kWriteThreads, s, false, d, per_head, static_cast<int>(items),
                  static_cast<const float*>(k), static_cast<const float*>(v), start, count, k8, ks, v8, vs, status);
  return launch(kvq_write_kernel<uint16_t>, dim3(grid), kWriteThreads, s, false, d, per_head, static_cast<int>(items),
                static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), start, count, k8, ks, v8, vs, status);
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
  const long long warps = static_cast<long long>(d.layers) * d.batch * d.n_kv_heads;
  const dim3 grid(static_cast<unsigned>((warps + 3) / 4));
  const int32_t* len = seq_len;
  cudaError_t e = d.dtype == EAGLE_F32
                      ? launch(kvq_commit_kernel<float>, grid, 128, s, true, d, a, n_acc, path, len, feat_cache, tree_feat)
                      : launch(kvq_commit_kernel<uint16_t>, grid, 128, s, true, d, a, n_acc, path, len, feat_cache,
                               tree_feat);
  if (e != cudaSuccess) return e;
  return launch_commit_finalize(d, n_acc, path, seq_len, commit_pos, status, s);
}

}  // namespace eagle
