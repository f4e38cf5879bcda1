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
// Bound by HBM for long inputs, by latency for one tree.  A warp takes one row, or a run of its
// heads when the rows alone would leave SMs empty (16 lanes x 8 elements = a head of 128, two
// heads a pass; four heads of 64), with three passes' loads in
// flight (a slot is loaded again as soon as its elements are in use).  Warps need nothing of one
// another, so one warp's loads, another's sines and a third's stores overlap: 46 us for 8192 rows
// of 48 heads (201 MB, 4.37 TB/s, 64 % of a large copy's rate; in fp32 72 us, 83 %).  A CTA per row with
// the sines shared over its heads took 76 us, every CTA going through its load, barrier and store
// phases alone.  The row's rot / 2 sines and cosines are computed two a lane into the warp's table
// while the first loads are on their way to L2.
// The angle is reduced in fp64 turns (pos * inv_freq / 2 pi, minus the nearest integer): in fp32
// the product alone would be off by 2^-24 of the angle, 4e-3 rad at position 65536.  Everything
// else is fp32, rounded once.
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace eagle {
namespace {

using sm100::f32x2_split;
using sm100::fma_f32x2;

constexpr int kThreads = 128;

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return sm100::f32x2(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

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
  int run, runs;  // heads a warp takes, runs of them in a row
  int units;
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
  // the elements that lane `src` of the group holds
  __device__ __forceinline__ Lane8 from(int src, int width) const {
    Lane8 r;
    r.u.x = __shfl_sync(0xffffffffu, u.x, src, width);
    r.u.y = __shfl_sync(0xffffffffu, u.y, src, width);
    r.u.z = __shfl_sync(0xffffffffu, u.z, src, width);
    r.u.w = __shfl_sync(0xffffffffu, u.w, src, width);
    return r;
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
  __device__ __forceinline__ Lane8 from(int src, int width) const {
    Lane8 r;
    float f[8];
    get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __shfl_sync(0xffffffffu, f[e], src, width);
    r.a = make_float4(f[0], f[1], f[2], f[3]);
    r.b = make_float4(f[4], f[5], f[6], f[7]);
    return r;
  }
  static __device__ __forceinline__ void store(void* p, size_t e, const float (&f)[8]) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
    d[0] = make_float4(f[0], f[1], f[2], f[3]);
    d[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <bool F32, int D>
__global__ void __launch_bounds__(kThreads, F32 ? 5 : 7) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int LANES = D / 8;       // lanes of a head
  constexpr int HPP = 32 / LANES;    // heads of a pass
  constexpr int U = F32 ? 2 : 3;     // passes whose loads are in flight together
  __shared__ __align__(16) float2 table[kThreads / 32][D / 2];
  const int warp = threadIdx.x >> 5;
  const int unit = blockIdx.x * (kThreads / 32) + warp;
  if (unit >= a.units) return;
  const int row32 = unit / a.runs, b = row32 / a.rows, r = row32 % a.rows;
  const size_t row = static_cast<size_t>(row32);
  if (a.n_nodes && r >= a.n_nodes[b]) return;  // rows past the request's tree are not written
  const int sub = (threadIdx.x & 31) / LANES, lane = threadIdx.x % LANES;
  const int h_begin = (unit - row32 * a.runs) * a.run;
  const int h_end = min(h_begin + a.run, a.hq + 2 * a.hkv);
  const size_t src = row * a.stride + static_cast<size_t>(lane) * 8;
  if (h_begin + sub < h_end)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(a.qkv) +
                                                  (src + static_cast<size_t>(h_begin + sub) * D) * (F32 ? 4 : 2)));
  const int half = a.rot / 2;
  const double pos = static_cast<double>(a.pos[row]) * 0.15915494309189533577;  // 1 / (2 pi)
  for (int i = threadIdx.x & 31; i < half; i += 32) {
    const double turns = pos * static_cast<double>(a.inv_freq[i]);
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    table[warp][i] = make_float2(c, s);
  }
  __syncwarp();
  // y = g (x c + p s): g the head's norm, p the rotation partner, c and s the lane's 8 cosines
  // and signed sines times the norm weights of x and p (reloaded when the heads turn from q to
  // k).  In the split form all 8 elements are first or all second ones (rot is a multiple of 16)
  // and a lane rot / 16 away has the partners; interleaved they are neighbours within the lane.
  const bool in = lane * 8 < a.rot;
  const bool second = !a.interleaved && lane * 8 >= half;
  const int far = !in || a.interleaved ? 0 : (second ? -(half / 8) : half / 8);
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {  // q, k, v heads of the run
    const int first = kind == 0 ? 0 : (kind == 1 ? a.hq : a.hq + a.hkv);
    const int k0 = max(h_begin, first), k1 = min(h_end, kind == 0 ? a.hq : first + a.hkv);
    if (k0 >= k1) continue;
    Lane8<F32> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = k0 + u * HPP + sub;
      if (h < k1) x[u].load(a.qkv, src + static_cast<size_t>(h) * D);
    }
    const void* weight = kind == 0 ? a.wq : (kind == 1 ? a.wk : nullptr);
    uint64_t c2[4], s2[4];  // in pairs
    if (kind < 2) {
      float c[8], s[8];
      Lane8<F32> t;
      float w[8], wp[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
      if (weight) {
        t.load(weight, static_cast<size_t>(lane) * 8);
        t.get(w);
        t.load(weight, static_cast<size_t>(lane + far) * 8);
        t.get(wp);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float2 v = make_float2(1.f, 0.f);
        if (in) v = table[warp][a.interleaved ? lane * 4 + e / 2 : lane * 8 + e - (second ? half : 0)];
        c[e] = w[e] * v.x;
        s[e] = (a.interleaved ? w[e ^ 1] : wp[e]) * ((a.interleaved ? (e & 1) != 0 : second) ? v.y : -v.y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c2[e] = pair(c[2 * e], c[2 * e + 1]);
        s2[e] = pair(s[2 * e], s[2 * e + 1]);
      }
    }
    // this lane's 16 bytes (bf16) of head h in the output of its kind
    uint8_t* out = static_cast<uint8_t*>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v));
    const size_t head0 = kind == 0 ? row * a.hq : static_cast<size_t>(b) * a.hkv * a.rows + r;
    const size_t step = kind == 0 ? 1 : a.rows;
    for (int h0 = k0; h0 < k1; h0 += U * HPP) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * HPP + sub;
        if (h - sub >= k1) break;  // the same for the whole warp: the shuffles below are warp-wide
        float f[8];
        x[u].get(f);
        if (kind < 2) {
          // two elements an instruction from here on
          uint64_t f2[4], p2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f2[e] = pair(f[2 * e], f[2 * e + 1]);
          if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) p2[e] = pair(f[2 * e + 1], f[2 * e]);
          } else {
            float p[8];
            x[u].from(lane + far, LANES).get(p);
#pragma unroll
            for (int e = 0; e < 4; ++e) p2[e] = pair(p[2 * e], p[2 * e + 1]);
          }
          float g = 1.f;
          if (weight) {
            uint64_t ss2 = mul_f32x2(f2[0], f2[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) ss2 = fma_f32x2(f2[e], f2[e], ss2);
            float s0, s1;
            f32x2_split(ss2, s0, s1);
            float ss = s0 + s1;
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, LANES);
            g = rsqrtf(ss * (1.f / D) + a.eps);
          }
          const uint64_t g2 = pair(g, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (the elements that do not turn have no partner: infinities times their sine of 0)
            const uint64_t t = mul_f32x2(f2[e], c2[e]);
            f32x2_split(mul_f32x2(in ? fma_f32x2(p2[e], s2[e], t) : t, g2), f[2 * e], f[2 * e + 1]);
          }
        }
        const int next = h + U * HPP;  // the slot's next head
        if (next < k1) x[u].load(a.qkv, src + static_cast<size_t>(next) * D);
        if (h < k1) Lane8<F32>::store(out, (head0 + (h - first) * step) * D + lane * 8, f);
      }
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const eagle_qk_norm_rope_desc& d, const void* qkv, const void* wq, const void* wk,
                                const float* inv_freq, const int32_t* pos_id, const int32_t* n_nodes, void* q,
                                void* k, void* v, int num_sms, cudaStream_t s) {
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
  // a whole row to a warp when that makes 16 warps an SM or more, else shorter runs of heads
  // (whole passes of 128 / D x 2 heads)
  const int heads = d.n_q_heads + 2 * d.n_kv_heads, pass = 256 / d.head_dim;
  const long long rows = static_cast<long long>(d.rows) * d.batch;
  const long long want = 16ll * num_sms;
  long long split = std::min<long long>((want + rows - 1) / rows, (heads + pass - 1) / pass);
  a.run = static_cast<int>(((heads + split - 1) / split + pass - 1) / pass * pass);
  a.runs = (heads + a.run - 1) / a.run;
  a.units = static_cast<int>(rows * a.runs);
  const int grid = (a.units + kThreads / 32 - 1) / (kThreads / 32);
  const bool f32 = d.dtype == EAGLE_F32;
  if (d.head_dim == 64)
    f32 ? qk_norm_rope_kernel<true, 64><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a)
        : qk_norm_rope_kernel<false, 64><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
  else
    f32 ? qk_norm_rope_kernel<true, 128><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a)
        : qk_norm_rope_kernel<false, 128><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace eagle
