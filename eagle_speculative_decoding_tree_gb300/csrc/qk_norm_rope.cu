// qk_norm_rope.cu -- from the QKV projection's rows to tree attention's operands: the norm
// of each query and key head, the rotation at each node's position, and the layout change,
// in one pass.
//
// For one head x of D elements (norm only with a weight w):
//     y = x / sqrt(mean(x^2) + eps) * w
//     (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = pos * inv_freq[i]
// over the first rot elements, a pair being (i, i + rot / 2) or (2 i, 2 i + 1).  A tree
// node's position is its prefix length plus its depth (pos_id of the tree build), so the
// nodes of one row block sit at few distinct positions, in no order.
//
// Bound by HBM for long inputs, by latency for one tree.  One CTA per row: its 16 half-warps
// take the Hq + 2 Hkv heads in turn (16 lanes x 8 elements = a head of 128; two heads of 64),
// the loads of the first heads are in flight while the row's rot / 2 sines and cosines are
// computed once, into shared memory, for every head.  The angle is reduced in fp64 turns
// (pos * inv_freq / 2 pi, minus the nearest integer): in fp32 the product alone would be off
// by 2^-24 of the angle, 4e-3 rad at position 65536.  Everything else is fp32, rounded once.
#include "common.cuh"
#include "launch.h"

namespace eagle {
namespace {

constexpr int kThreads = 256;

struct RopeArgs {
  const void* qkv;
  const void* wq;
  const void* wk;
  const float* inv_freq;
  const int32_t* pos;
  const int32_t* n_nodes;
  void* q;
  void* k;
  void* v;
  int rows, hq, hkv, rot, interleaved;
  long long stride;
  float eps;
};

template <bool F32>
struct Lane8;  // a lane's 8 consecutive elements
template <>
struct Lane8<false> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p, size_t e) {
    u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, size_t e, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Lane8<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, size_t e) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    a = __ldg(s);
    b = __ldg(s + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, size_t e, const float (&f)[8]) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
    d[0] = make_float4(f[0], f[1], f[2], f[3]);
    d[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <bool F32, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int LANES = D / 8;              // lanes of a head
  constexpr int GROUPS = kThreads / LANES;  // heads of a CTA pass
  constexpr int U = 4;                      // passes whose loads are in flight together
  __shared__ float2 cs[D / 2];
  const int b = blockIdx.y, r = blockIdx.x;
  if (a.n_nodes && r >= a.n_nodes[b]) return;  // rows past the request's tree are not written
  const int grp = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int heads = a.hq + 2 * a.hkv;
  const size_t row = static_cast<size_t>(b) * a.rows + r;
  const size_t src = row * a.stride + static_cast<size_t>(lane) * 8;
  Lane8<F32> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (grp + u * GROUPS < heads) x[u].load(a.qkv, src + static_cast<size_t>(grp + u * GROUPS) * D);
  const int half = a.rot / 2;
  if (threadIdx.x < half) {
    const double turns = static_cast<double>(a.pos[row]) * static_cast<double>(a.inv_freq[threadIdx.x]) *
                         0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    cs[threadIdx.x] = make_float2(c, s);
  }
  float w[2][8];  // the lane's norm weights of q and k
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const void* p = t ? a.wk : a.wq;
    Lane8<F32> y;
    if (p) {
      y.load(p, static_cast<size_t>(lane) * 8);
      y.get(w[t]);
    }
  }
  __syncthreads();
  // the lane's 8 rotation pairs: in the split form all of them are first or all second
  // elements (rot is a multiple of 16), whose partners a lane rot / 16 away holds
  const bool in = lane * 8 < a.rot;
  const bool second = !a.interleaved && lane * 8 >= half;
  const int far = !in || a.interleaved ? 0 : (second ? -(half / 8) : half / 8);
  for (int h0 = grp; h0 - grp < heads; h0 += U * GROUPS) {
    if (h0 != grp) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h0 + u * GROUPS < heads) x[u].load(a.qkv, src + static_cast<size_t>(h0 + u * GROUPS) * D);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * GROUPS;
      if (h - grp >= heads) break;  // the same for the whole CTA: the shuffles below are warp-wide
      const bool live = h < heads;
      const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
      float f[8];
      x[u].get(f);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, LANES);
      if (is_q ? a.wq != nullptr : (is_k && a.wk != nullptr)) {
        const float g = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= g * (is_q ? w[0][e] : w[1][e]);
      }
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(0xffffffffu, f[e], lane + far, LANES);
      if ((is_q || is_k) && in) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 t = cs[lane * 4 + e];
            const float u0 = f[2 * e], u1 = f[2 * e + 1];
            f[2 * e] = u0 * t.x - u1 * t.y;
            f[2 * e + 1] = u0 * t.y + u1 * t.x;
          }
        } else {
          const int i0 = lane * 8 - (second ? half : 0);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 t = cs[i0 + e];
            f[e] = second ? p[e] * t.y + f[e] * t.x : f[e] * t.x - p[e] * t.y;
          }
        }
      }
      if (!live) continue;
      if (is_q) {
        Lane8<F32>::store(a.q, (row * a.hq + h) * D + lane * 8, f);
      } else {
        const int kh = h - a.hq - (is_k ? 0 : a.hkv);
        Lane8<F32>::store(is_k ? a.k : a.v,
                          ((static_cast<size_t>(b) * a.hkv + kh) * a.rows + r) * D + lane * 8, f);
      }
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const eagle_qk_norm_rope_desc& d, const void* qkv, const void* wq, const void* wk,
                                const float* inv_freq, const int32_t* pos_id, const int32_t* n_nodes, void* q,
                                void* k, void* v, cudaStream_t s) {
  RopeArgs a;
  a.qkv = qkv;
  a.wq = wq;
  a.wk = wk;
  a.inv_freq = inv_freq;
  a.pos = pos_id;
  a.n_nodes = n_nodes;
  a.q = q;
  a.k = k;
  a.v = v;
  a.rows = d.rows;
  a.hq = d.n_q_heads;
  a.hkv = d.n_kv_heads;
  a.rot = d.rot_dim;
  a.interleaved = d.interleaved;
  a.stride = d.row_stride > 0 ? d.row_stride : static_cast<long long>(d.n_q_heads + 2 * d.n_kv_heads) * d.head_dim;
  a.eps = d.eps;
  const dim3 grid(d.rows, d.batch);
  const bool f32 = d.dtype == EAGLE_F32;
  if (d.head_dim == 64)
    f32 ? qk_norm_rope_kernel<true, 64><<<grid, kThreads, 0, s>>>(a)
        : qk_norm_rope_kernel<false, 64><<<grid, kThreads, 0, s>>>(a);
  else
    f32 ? qk_norm_rope_kernel<true, 128><<<grid, kThreads, 0, s>>>(a)
        : qk_norm_rope_kernel<false, 128><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace eagle
