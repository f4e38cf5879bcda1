// tree_attn_kvq_tc.cu -- tree attention over the 8-bit KV cache on the tcgen05 tensor cores
// (head_dim 128), for trees of many rows; tree_attn_kvq.cu has the operation and the
// few-row kernel.
//
// Q K^T takes the codes as they come: kind::f8f6f4.  A query row is multiplied by a power of two
// and split into terms of three or four bits that hold bf16's eight (kvq_split2, kvq_split3): two,
// exact down to elements of 2^-13 of the row's largest, or for EAGLE_ATTN_PRECISE three, exact down
// to 2^-23 of it.  Two products at twice the half rate cost what one half product would, and K is
// never converted.  P V takes halves (11 bits in one term, against
// the four of an e4m3 P): six warps widen each V tile from e4m3 to half, exactly, into a
// second ring.  The scales stay outside as in tree_attn_kvq.cu: ks on the scores of its 64
// keys, vs / vref in the exponent of P.
//
// One CTA per (piece, request x KV head, row block), 512 threads:
//   warps 0-3, 4-7  softmax warpgroups; a thread owns one row (its TMEM lane) and a tile's 128
//                   scores.  With one term of P it takes them in one pass: exponentials against
//                   the row's reference as it stands, P in registers until the maximum has
//                   confirmed the reference; else (first tiles, masked tiles, two terms) in two
//                   passes, maximum first.
//   warps 8-13      V widening.
//   warp 14         TMA producer of the two code rings.
//   warp 15         issues every tcgen05.mma: QK0 QK1 | PV0 QK2 | PV1 QK3 | ...
// Items alternate between the warpgroups, so one tile's products run under the other's softmax.
// With 256 rows a CTA (A) warpgroup w has rows 128 w .. and both take every tile: the codes are
// read and widened once for 256 rows.  With 128 (B; up to 128 rows a KV head, and more over short
// prefixes: plan_kvq_attn) both have the same rows and take alternate tiles; their states merge in
// the epilogue.
// TMEM: S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512); P overwrites S in place.
//
// Piece 0 is the tree itself (bf16 Q and K, V and P in halves, P always in two terms, one tile);
// the others are tps 128-key tiles of the prefix.  Pieces write fp32 partials (TMA stores).  When the
// whole grid fits on the SMs the launch is cooperative and the pieces of a group merge their rows
// in the kernel (a second launch costs several microseconds); otherwise kvq_combine_kernel does.
//
// Bound by the products and the chain S -> P -> PV -> next S (P takes S's place in TMEM): 2690
// cycles for 256 rows x 128 keys against 2048 of products (two e4m3 ones and one half one, 64
// cycles per 128 x 128 x 32 bytes).  Measured, graph replay, FAST (PRECISE): 61 nodes x 4 heads x 8 over
// 128K 112 us (144), 1170 TFLOP/s, over 8K 19.1 us (21.1; half of it staging, partials and merge), 32
// requests of 1K to 16K 262 us (348).
#include "common.cuh"
#include "kvq.cuh"
#include "kvq_merge.cuh"
#include "launch.h"
#include "sm100.cuh"
#include "tmap.h"

namespace eagle {
namespace {

using namespace sm100;

constexpr int KT = 128;
constexpr int T8 = KT * 128;    // a tile of codes, 16 KB
constexpr int T16 = 2 * T8;     // a tile of halves, 32 KB: two 64-dim halves of 128-byte rows
// Shared memory by terms of P (EAGLE_ATTN_FAST 1, PRECISE 2): two row tiles of Q's terms (or bf16
// halves), the rings of K and V codes, widened V (two stages).  The third term of Q takes a stage of
// either ring.
template <int TERMS>
struct Lay {
  static constexpr int QT = TERMS == 2 ? 3 : 2;   // terms of Q
  static constexpr int KST = TERMS == 2 ? 2 : 3, VST = KST;
  static constexpr int QB = QT * T8;              // a row tile's Q
  static constexpr int SM_Q = 0;
  static constexpr int SM_K = SM_Q + 2 * QB;
  static constexpr int SM_V = SM_K + KST * T8;
  static constexpr int SM_W = SM_V + VST * T8;
  static constexpr int SMEM = SM_W + 2 * T16 + 1024;
};
constexpr int NT = 512;
constexpr int WT = 192;                 // widening threads (six warps)
constexpr int QW = 14;                  // warps that stage the query tile: softmax and widening
constexpr float kLazy = 4.f;            // as in tree_attn_kvq.cu
constexpr int PB = 11;

enum : int { ERR_K = 1, ERR_KE = 2, ERR_V = 4, ERR_W = 8, ERR_WE = 16, ERR_S = 32, ERR_P = 64, ERR_O = 128, ERR_GROUP = 256, ERR_Q = 512,
             ERR_VE = 1024 };

struct Maps {
  CUtensorMap k, v, po;
};

__device__ __forceinline__ uint32_t col_s(int w) { return static_cast<uint32_t>(w) * 128u; }
__device__ __forceinline__ uint32_t col_o(int w) { return 256u + static_cast<uint32_t>(w) * 128u; }

// Instruction descriptors: fp32 accumulator; operand formats in bits 7 and 10 (f8f6f4: e4m3 0, e5m2 1;
// f16: half 0, bf16 1).
__host__ __device__ constexpr uint32_t idesc(int fmt, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(fmt) << 7) | (static_cast<uint32_t>(fmt) << 10) |
         (static_cast<uint32_t>(b_mn) << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}

// tcgen05.mma and commit by one elected lane of a converged warp: the whole warp computes the
// descriptors, so they stay in uniform registers.  (Issued from a lane == 0 branch each product
// took about 150 cycles to issue, more than it runs.)
__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(at), "l"(bd), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float max32(const uint32_t (&a)[32]) {
  float m[11];
#pragma unroll
  for (int i = 0; i < 10; ++i)
    m[i] = max3(__uint_as_float(a[3 * i]), __uint_as_float(a[3 * i + 1]), __uint_as_float(a[3 * i + 2]));
  m[10] = fmaxf(__uint_as_float(a[30]), __uint_as_float(a[31]));
  return fmaxf(max3(max3(m[0], m[1], m[2]), max3(m[3], m[4], m[5]), max3(m[6], m[7], m[8])), fmaxf(m[9], m[10]));
}

__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// 32 scores -> P in columns col .. (TERMS 1: 16 of them, TERMS 2: hi 16, lo 16), p = 2^(s c + o);
// unless FULL, keys whose bit is clear get 0.  Returns the fp32 sum.
template <int TERMS, bool FULL>
__device__ __forceinline__ float emit(const uint32_t (&r)[32], uint32_t col, float c, float o, uint32_t bits) {
  const uint64_t c2 = f32x2(__float_as_uint(c), __float_as_uint(c)), o2 = f32x2(__float_as_uint(o), __float_as_uint(o));
  uint64_t acc = 0ull;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = 16 * g + 2 * j;
      float x0, x1;
      f32x2_split(fma_f32x2(f32x2(r[k], r[k + 1]), c2, o2), x0, x1);
      float p0 = ex2(x0), p1 = ex2(x1);
      if (!FULL) {
        p0 = (bits >> k) & 1u ? p0 : 0.f;
        p1 = (bits >> (k + 1)) & 1u ? p1 : 0.f;
      }
      acc = add_f32x2(acc, f32x2(__float_as_uint(p0), __float_as_uint(p1)));
      hi[j] = half2_bits(p0, p1);
      if (TERMS == 2) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
        lo[j] = half2_bits(p0 - f.x, p1 - f.y);
      }
    }
    tmem_st8(col + 8 * g, hi);
    if (TERMS == 2) tmem_st8(col + 16 + 8 * g, lo);
  }
  float a0, a1;
  f32x2_split(acc, a0, a1);
  return a0 + a1;
}

// 32 scores -> P as 16 packed halves, p = 2^(s c + o); returns the fp32 sum.
__device__ __forceinline__ float to_half(const uint32_t (&r)[32], uint32_t (&p)[32], int at, float c, float o) {
  const uint64_t c2 = f32x2(__float_as_uint(c), __float_as_uint(c)), o2 = f32x2(__float_as_uint(o), __float_as_uint(o));
  uint64_t acc = 0ull;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float x0, x1;
    f32x2_split(fma_f32x2(f32x2(r[2 * j], r[2 * j + 1]), c2, o2), x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    acc = add_f32x2(acc, f32x2(__float_as_uint(p0), __float_as_uint(p1)));
    p[at + j] = half2_bits(p0, p1);
  }
  float a0, a1;
  f32x2_split(acc, a0, a1);
  return a0 + a1;
}

// row / G for row G < 2^32: a multiplication by ceil(2^32 / G) (a division costs as much as the
// rest of a row's staging).
__device__ __forceinline__ int node_of(const KvqAttnArgs& a, int row) {
  return a.G == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), a.g_inv));
}

struct Range {
  int L, Rb, tile0, n;  // the piece's prefix tiles [tile0, tile0 + n); n = 1 for the tree
  bool tree;
};

template <int TERMS>
__global__ void __launch_bounds__(NT, 1) tree_attn_kvq_tc_kernel(const __grid_constant__ Maps tm, const KvqAttnArgs a) {
  using Y = Lay<TERMS>;
  constexpr int KST = Y::KST, VST = Y::VST, QB = Y::QB, SM_Q = Y::SM_Q, SM_K = Y::SM_K, SM_V = Y::SM_V, SM_W = Y::SM_W;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t k_full[KST], k_empty[KST], v_full[VST], v_empty[VST], w_full[2], w_empty[2], s_full[2], p_full[2], q_full, o_full;
  __shared__ uint32_t tmem_base;
  __shared__ int go;             // group merge: every piece counted in time
  __shared__ float s_q[2][128];  // the query rows' factors; tree: [0][0] the unit of V's halves
  // row maxima and sums of the two warpgroups, exchanged in the epilogue (the widened V's area,
  // free by then)
  float (*s_m)[128] = reinterpret_cast<float (*)[128]>(smem + SM_W);
  float (*s_l)[128] = reinterpret_cast<float (*)[128]>(smem + SM_W + 1024);

  // Dispatch order.  One wave: a group's pieces next to each other.  Else every request's first
  // prefix piece, then the second ones, ...: full pieces come before the shorter last ones of
  // ragged requests, and the trees, the shortest, fill the end (row blocks of one piece, which
  // read the same codes, next to each other).
  int piece, bh, rb;
  kvq_place(a, a.rows_pad / (a.wr * 128), piece, bh, rb);
  const int b = bh / a.Hkv, h = bh % a.Hkv;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int row0 = rb * a.wr * 128;

  if (warp == 15) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < KST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], WT / 32);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&w_full[s], WT / 32);
      mbar_init(&w_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 128);
    }
    mbar_init(&q_full, QW);
    mbar_init(&o_full, 1);
    fence_barrier_init();
  }
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();

  Range r;
  r.L = a.seq_len[b];
  r.L = r.L < 0 ? 0 : (r.L > a.P ? a.P : r.L);
  r.Rb = a.n_nodes ? min(max(a.n_nodes[b], 0), a.R) : a.R;
  r.tree = piece == 0;
  const int n_pref = (r.L + KT - 1) / KT;
  const int tps = kvq_tps(a, n_pref);
  r.tile0 = (piece - 1) * tps;
  r.n = r.tree ? 1 : max(0, min(tps, n_pref - r.tile0));
  const int RG = r.Rb * a.G;
  const bool two = a.wr == 2 && RG - row0 > 128;  // A: two row tiles
  const bool work = r.n > 0 && row0 < RG;
  const int items = work ? (two ? 2 * r.n : r.n) : 0;
  auto tile_of = [&](int i) { return two ? i >> 1 : i; };
  auto last_of = [&](int i) { return !two || (i & 1); };  // the tile's last item
  const uint32_t tb = tmem_base;
  const int nblk = (a.P + kQB - 1) / kQB;

  if (warp < QW && work) {
    // ------------------------------------------------------------ Q: four rows at a time, eight lanes a row
    // All copies are asynchronous, 128 bytes of a row by its eight lanes: dims 8 c .. and 64 + 8 c ..
    // in swizzled rows of 64 bf16 dims.  That is the tree's final form; a prefix piece's codes (128 to
    // a row) then replace them in place: every warp that would wait takes part (61 nodes over 2K, one
    // query head a KV head: 15.5 us, 16.7 by the softmax warps alone).
    // (Loops rolled: straight-line code that runs once costs its instruction fetches.)
    const int c = lane & 7, sub = lane >> 3, units = two ? 64 : 32;
    const uint32_t d0 = smem_u32(smem + SM_Q);
#pragma unroll 1
    for (int u = warp; u < units; u += QW) {
      const int lr = (u & 31) * 4 + sub, qr = row0 + u * 4 + sub;
      const int nd = node_of(a, qr), n16 = qr < RG ? 16 : 0;  // 0: zero fill, nothing read
      const uint16_t* src =
          n16 ? a.q + ((static_cast<size_t>(b) * a.R + nd) * a.Hq + h * a.G + (qr - nd * a.G)) * 128 + 8 * c : a.q;
      const uint32_t at = d0 + (u >> 5) * QB + lr * 128 + ((c ^ (lr & 7)) << 4);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(src), "r"(n16) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + T8), "l"(src + 64), "r"(n16) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
#pragma unroll 1
    for (int u = warp; u < units && !r.tree; u += QW) {
      const int lr = (u & 31) * 4 + sub;
      uint8_t* dst = smem + SM_Q + (u >> 5) * QB;
      if (row0 + u * 4 >= RG) {  // zeros in either form
        if (TERMS == 2) *reinterpret_cast<uint4*>(dst + 2 * T8 + lr * 128 + c * 16) = make_uint4(0, 0, 0, 0);
        if (c == 0) s_q[u >> 5][lr] = 1.f;
        continue;
      }
      const uint8_t* d = dst + lr * 128 + ((c ^ (lr & 7)) << 4);
      const uint4 x0 = *reinterpret_cast<const uint4*>(d), x1 = *reinterpret_cast<const uint4*>(d + T8);
      const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
      uint32_t am = 0;  // the row's largest magnitude, as bf16 bits (ordered as integers)
#pragma unroll
      for (int k = 0; k < 8; ++k) am = max(am, max((x[k] << 16) & 0x7fff0000u, x[k] & 0x7fff0000u));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
      // a row with an element that is not finite gets NaN scores
      const float qs = kvq_qscale(am, TERMS == 2);
      const float mul = __uint_as_float((254u << 23) - __float_as_uint(qs));  // 1 / qs, a power of two
      if (c == 0) s_q[u >> 5][lr] = am < 0x7f800000u ? qs : __uint_as_float(0x7fffffffu);
      uint32_t tq[Y::QT][4];  // words 0, 1: dims 8 c ..; 2, 3: dims 64 + 8 c ..
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t t[2][3];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t v = x[2 * k + e];
          const uint32_t h = half2_bits(__uint_as_float(v << 16) * mul, __uint_as_float(v & 0xffff0000u) * mul);
          if (TERMS == 2)
            kvq_split3(h, t[e]);
          else
            kvq_split2<false>(h, t[e][0], t[e][1]);
        }
#pragma unroll
        for (int i = 0; i < Y::QT; ++i) tq[i][k] = kvq_pack(t[0][i], t[1][i]);
      }
      // (every lane of the row has its elements: the maximum's shuffles came between)
      uint8_t* d1 = dst + lr * 128 + (((c >> 1) ^ (lr & 7)) << 4) + 8 * (c & 1);
      uint8_t* d2 = dst + lr * 128 + ((((c >> 1) + 4) ^ (lr & 7)) << 4) + 8 * (c & 1);
#pragma unroll
      for (int i = 0; i < Y::QT; ++i) {
        *reinterpret_cast<uint2*>(d1 + i * T8) = make_uint2(tq[i][0], tq[i][1]);
        *reinterpret_cast<uint2*>(d2 + i * T8) = make_uint2(tq[i][2], tq[i][3]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full);
  }

  // registers: 128 a thread at launch (65536); the softmax takes 176 each, the others keep 80
  // (256 x 176 + 256 x 80 = 65536)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 14) {
      // ------------------------------------------------------------ TMA producer (lane 0)
      if (lane == 0 && work && !r.tree) {
        const uint64_t policy = policy_evict_first();
        const int y0 = bh * a.P + r.tile0 * KT;
        auto load = [&](const CUtensorMap& m, int at, uint64_t* bar, int t) {
          mbar_arrive_expect_tx(bar, T8);
          tma_load_2d_hint(smem + at, &m, 0, y0 + t * KT, bar, policy);
        };
        int k_in = 0, v_in = 0;  // loads issued
        for (int t = 0; t < r.n; ++t) {
          const int s = t % KST, sv = t % VST;
          if (t >= KST && !wait_parity(&k_empty[s], (t / KST - 1) & 1, a.err, ERR_KE)) break;
          load(tm.k, SM_K + s * T8, &k_full[s], t);
          ++k_in;
          if (t >= VST && !wait_parity(&v_empty[sv], (t / VST - 1) & 1, a.err, ERR_VE)) break;
          load(tm.v, SM_V + sv * T8, &v_full[sv], t);
          ++v_in;
          // the first tile first: with the whole ring's loads ahead of it the query tile would
          // arrive last, and nothing can start without it
          if (t == 0 && !wait_parity(&q_full, 0, a.err, ERR_Q)) break;
        }
        // no copy may still be landing when the CTA ends
        for (int s = 0; s < KST && s < k_in; ++s) (void)wait_parity(&k_full[s], ((k_in - 1 - s) / KST) & 1, a.err, ERR_K);
        for (int s = 0; s < VST && s < v_in; ++s) (void)wait_parity(&v_full[s], ((v_in - 1 - s) / VST) & 1, a.err, ERR_V);
      }
    } else if (warp >= 8 && warp < 14) {
      // ------------------------------------------------------------ V widening
      const int id = threadIdx.x - 256;
      if (work && !r.tree) {
        for (int t = 0; t < r.n; ++t) {
          const int s = t % VST, w = t & 1;
          bool ok = wait_parity(&v_full[s], (t / VST) & 1, a.err, ERR_V);
          if (ok && t >= 2) ok = wait_parity(&w_empty[w], ((t >> 1) - 1) & 1, a.err, ERR_WE);
          if (!__all_sync(0xffffffffu, ok)) break;
          const int nv = min(KT, r.L - (r.tile0 + t) * KT);
          const uint8_t* src = smem + SM_V + s * T8;
          uint8_t* dst = smem + SM_W + w * T16;
          // 16 codes at a time; all of a thread's loads first (the stores could alias them)
          constexpr int N = (KT * 8 + WT - 1) / WT;
          uint4 u[N];
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int i = id + WT * e, row = i & 127;
            u[e] = make_uint4(0, 0, 0, 0);  // rows past the prefix: zeros, whatever they hold
            if (i < KT * 8 && row < nv)
              u[e] = *reinterpret_cast<const uint4*>(src + row * 128 + (((i >> 7) ^ (row & 7)) << 4));
          }
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int i = id + WT * e, row = i & 127, c = i >> 7, p = 2 * (c & 3);
            if (i >= KT * 8) break;
            uint8_t* d = dst + (c >> 2) * T8 + row * 128;
            *reinterpret_cast<uint4*>(d + ((p ^ (row & 7)) << 4)) =
                make_uint4(kvq_half2(u[e].x), kvq_half2(u[e].x >> 16), kvq_half2(u[e].y), kvq_half2(u[e].y >> 16));
            *reinterpret_cast<uint4*>(d + (((p + 1) ^ (row & 7)) << 4)) =
                make_uint4(kvq_half2(u[e].z), kvq_half2(u[e].z >> 16), kvq_half2(u[e].w), kvq_half2(u[e].w >> 16));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&w_full[w]);
            mbar_arrive(&v_empty[s]);
          }
        }
      } else if (work) {
        // The tree's K tile as it is (bf16); its V as halves, times the power of two that puts the
        // tile's largest element in [2^14, 2^15): exact for elements down to 2^-32 of that one,
        // in steps of 2^-39 of it below.  Zeros behind the tree's rows.
        const uint4* kg = reinterpret_cast<const uint4*>(a.tk + static_cast<size_t>(bh) * a.R * 128);
        const uint4* vg = reinterpret_cast<const uint4*>(a.tv + static_cast<size_t>(bh) * a.R * 128);
        constexpr int U = 6;  // 16-byte pieces of a thread in flight (two rounds above 72 rows)
        auto at = [&](int i) {
          const int row = i >> 4, c = i & 15;
          return (c >> 3) * T8 + row * 128 + (((c & 7) ^ (row & 7)) << 4);
        };
        auto load = [&](uint4 (&x)[U], const uint4* g, int i0) {
#pragma unroll
          for (int e = 0; e < U; ++e) {
            x[e] = make_uint4(0, 0, 0, 0);
            if (i0 + e * WT < r.Rb * 16) x[e] = __ldg(g + i0 + e * WT);
          }
        };
        uint32_t am = 0;  // the largest finite magnitude of V, as float bits (ordered as integers)
        uint4 x[U];
#pragma unroll 1
        for (int i0 = id; i0 < KT * 16; i0 += U * WT) {
          uint4 k[U];
          load(x, vg, i0);
          load(k, kg, i0);
#pragma unroll
          for (int e = 0; e < U; ++e) {
            const uint32_t u[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const uint32_t p0 = (u[f] << 16) & 0x7fff0000u, p1 = u[f] & 0x7fff0000u;
              am = max(am, max(p0 < 0x7f800000u ? p0 : 0u, p1 < 0x7f800000u ? p1 : 0u));
            }
            if (i0 + e * WT < KT * 16) *reinterpret_cast<uint4*>(smem + SM_K + at(i0 + e * WT)) = k[e];
          }
        }
        am = __reduce_max_sync(0xffffffffu, am);
        if (lane == 0) s_q[1][warp - 8] = __uint_as_float(am);
        bar_sync(4, WT);
        for (int k = 0; k < WT / 32; ++k) am = max(am, __float_as_uint(s_q[1][k]));
        const int ex = max(static_cast<int>(am >> 23) - 127, -100);
        const float mul = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);
        if (id == 0) s_q[0][0] = __uint_as_float(static_cast<uint32_t>(127 + ex - 14) << 23);  // 1 / mul
        auto halves = [&](uint32_t u) {
          return half2_bits(__uint_as_float(u << 16) * mul, __uint_as_float(u & 0xffff0000u) * mul);
        };
#pragma unroll 1
        for (int n = (KT * 16 - 1) / (U * WT); n >= 0; --n) {  // (the last round's is still in registers)
          const int i0 = id + n * U * WT;
          if (n < (KT * 16 - 1) / (U * WT)) load(x, vg, i0);
#pragma unroll
          for (int e = 0; e < U; ++e)
            if (i0 + e * WT < KT * 16)
              *reinterpret_cast<uint4*>(smem + SM_W + at(i0 + e * WT)) =
                  make_uint4(halves(x[e].x), halves(x[e].y), halves(x[e].z), halves(x[e].w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_full[0]);
      }
    } else if (warp == 15) {
      // ------------------------------------------------------------ tcgen05.mma issue
      if (items > 0) {
        // every lane waits (and sees the same outcome): the warp stays converged for the elections
        auto wait = [&](uint64_t* bar, int parity, int code) {
          return __all_sync(0xffffffffu, wait_parity(bar, parity, a.err, code)) != 0;
        };
        const uint32_t tu = __shfl_sync(0xffffffffu, tb, 0);
        const int n = __shfl_sync(0xffffffffu, items, 0);
        const uint64_t dq = smem_desc_sw128(smem_u32(smem + SM_Q), 16, 1024);
        const uint64_t dk = smem_desc_sw128(smem_u32(smem + SM_K), 16, 1024);
        const uint64_t dv = smem_desc_sw128(smem_u32(smem + SM_W), T8, 1024);
        bool ok = wait(&q_full, 0, ERR_Q);
        if (r.tree) {
          ok = ok && wait(&w_full[0], 0, ERR_W);  // K and V both
          for (int w = 0; w < n && ok; ++w) {
            tc_fence_after();
#pragma unroll 1
            for (int ks = 0; ks < 8; ++ks) {
              const uint64_t off = (ks >> 2) * (T8 >> 4) + (ks & 3) * 2;
              mma_f16_ss(tu + col_s(w), dq + w * (QB >> 4) + off, dk + off, idesc(1, 0), ks > 0);
            }
            commit(&s_full[w]);
          }
          for (int w = 0; w < n && ok; ++w) {
            ok = wait(&p_full[w], 0, ERR_P);
            tc_fence_after();
#pragma unroll 1
            for (int ks = 0; ks < 8; ++ks) {  // hi 16 columns, lo 16
              const uint32_t ac = tu + col_s(w) + (ks >> 1) * 32 + (ks & 1) * 8;
              mma_f16_ts(tu + col_o(w), ac, dv + ks * 128, idesc(0, 1), ks > 0);
              mma_f16_ts(tu + col_o(w), ac + 16, dv + ks * 128, idesc(0, 1), 1u);
            }
          }
        } else {
          auto qk = [&](int i) {
            const int t = tile_of(i), w = i & 1, s = t % KST;
            // (A: the first row tile's item has waited for both; a wait costs what a product does)
            if ((!two || !w) && !wait(&k_full[s], (t / KST) & 1, ERR_K)) return false;
            tc_fence_after();
            const uint64_t q = dq + (two ? w * (QB >> 4) : 0), k = dk + s * (T8 >> 4);
#pragma unroll
            for (int term = 0; term < Y::QT; ++term)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)  // (the first of two terms is e4m3, as the codes; all others e5m2)
                mma_f8_ss(tu + col_s(w), q + term * (T8 >> 4) + ks * 2, k + ks * 2,
                          idesc(0, 0) | (TERMS == 2 || term ? 1u << 7 : 0u), term + ks > 0);
            commit(&s_full[w]);
            if (last_of(i)) commit(&k_empty[s]);
            return true;
          };
          auto pv = [&](int i) {
            const int t = tile_of(i), w = i & 1;
            if ((!two || !w) && !wait(&w_full[t & 1], (t >> 1) & 1, ERR_W)) return false;
            if (!wait(&p_full[w], (i >> 1) & 1, ERR_P)) return false;
            tc_fence_after();
            const uint64_t v = dv + (t & 1) * (T16 >> 4);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              // two terms: hi 16 columns, lo 16
              const uint32_t ac = tu + col_s(w) + (TERMS == 2 ? (ks >> 1) * 32 + (ks & 1) * 8 : ks * 8);
              mma_f16_ts(tu + col_o(w), ac, v + ks * 128, idesc(0, 1), (i >= 2 || ks > 0) ? 1u : 0u);
              if (TERMS == 2) mma_f16_ts(tu + col_o(w), ac + 16, v + ks * 128, idesc(0, 1), 1u);
            }
            if (last_of(i)) commit(&w_empty[t & 1]);
            return true;
          };
          ok = ok && qk(0) && (n < 2 || qk(1));
#pragma unroll 1
          for (int i = 0; i < n && ok; ++i) ok = pv(i) && (i + 2 >= n || qk(i + 2));
        }
        commit(&o_full);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    if (work) {
      // ------------------------------------------------------------ softmax
      const int w = warp >> 2, qd = warp & 3;
      const int rl = qd * 32 + lane;  // TMEM lane, row of the warpgroup's tile
      const int row = row0 + (two ? w * 128 : 0) + rl;
      const bool live = row < RG;
      const int node = live ? node_of(a, row) : 0;
      // vref: the largest V scale of the piece
      const float* ks = a.ks + static_cast<size_t>(bh) * nblk + r.tile0 * (KT / kQB);
      const float* vs = a.vs + static_cast<size_t>(bh) * nblk + r.tile0 * (KT / kQB);
      int n_blk = 0;
      float vref = 1.f;
      if (!r.tree) {
        n_blk = (min(r.L, (r.tile0 + r.n) * KT) + kQB - 1) / kQB - r.tile0 * (KT / kQB);
        float m = 0.f;
#pragma unroll 4
        for (int i = lane; i < n_blk; i += 32) m = fmaxf(m, __ldg(vs + i));
        vref = kvq_vref(warp_max(m));
      }
      const float vinv = 1.f / vref;
      // (orders every warp's s_q; a query tile that never came shows at the first scores)
      (void)wait_parity(&q_full, 0, a.err, ERR_Q);
      const float qs = r.tree ? 1.f : s_q[two ? w : 0][rl];
      uint32_t tw[4] = {0u, 0u, 0u, 0u};  // the tree's visible keys
      if (r.tree && live) {
        const uint64_t* mp = a.anc_mask + (static_cast<size_t>(b) * a.R + node) * a.W;
        const uint64_t w0 = mp[0], w1 = a.W > 1 ? mp[1] : 0ull;
        tw[0] = static_cast<uint32_t>(w0) & low_bits(r.Rb);
        tw[1] = static_cast<uint32_t>(w0 >> 32) & low_bits(r.Rb - 32);
        tw[2] = static_cast<uint32_t>(w1) & low_bits(r.Rb - 64);
        tw[3] = static_cast<uint32_t>(w1 >> 32) & low_bits(r.Rb - 96);
      }
      const float cr = a.scale_log2 * qs;
      const uint32_t lb = tb + (static_cast<uint32_t>(qd * 32) << 16);
      const uint32_t sc = lb + col_s(w), oc = lb + col_o(w);
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      float kn[2] = {0.f, 0.f}, vn[2] = {0.f, 0.f};  // the next tile's scales
      auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int kb = min(2 * t + u, n_blk - 1);
          kn[u] = __ldg(ks + kb);
          vn[u] = __ldg(vs + kb);
        }
      };
      if (!r.tree) fetch(min(tile_of(w), r.n - 1));
      for (int i = w; i < items; i += 2) {
        const int t = tile_of(i);
        float ck[2] = {cr, cr}, lr[2] = {PB, PB}, to[2] = {0.f, 0.f};
        if (!r.tree) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            ck[u] = cr * kn[u];
            lr[u] = kvq_ld(vn[u], vinv) + PB;
            to[u] = kvq_toward(lr[u] - PB);
          }
          fetch(min(tile_of(i + 2), r.n - 1));
        }
        const int nv = r.tree ? 0 : min(KT, r.L - (r.tile0 + t) * KT);
        uint32_t km[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) km[c] = r.tree ? tw[c] : low_bits(nv - 32 * c);
        const bool full = !r.tree && nv == KT;
        ok = __all_sync(0xffffffffu, wait_parity(&s_full[w], (i >> 1) & 1, a.err, ERR_S));
        if (!ok) break;
        tc_fence_after();
        uint32_t x[32], y[32];
        if (TERMS == 1 && full && i >= 2) {
          // One pass: the exponentials against the reference as it stands, P held in registers
          // until the maximum has confirmed it (nearly always, after the first tiles); otherwise
          // S is still there for the two passes below.
          uint32_t p0[32], p1[32];
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          tmem_ld32(sc, x);
          tmem_ld32(sc + 32, y);
          tmem_ld_wait();
          float mx = max32(x);
          float s0 = to_half(x, p0, 0, ck[0], lr[0] - mu);
          tmem_ld32(sc + 64, x);
          mx = fmaf(fmaxf(mx, max32(y)), ck[0], to[0]);
          s0 += to_half(y, p0, 16, ck[0], lr[0] - mu);
          tmem_ld_wait();
          tmem_ld32(sc + 96, y);
          float mz = max32(x);
          float s1 = to_half(x, p1, 0, ck[1], lr[1] - mu);
          tmem_ld_wait();
          mz = fmaf(fmaxf(mz, max32(y)), ck[1], to[1]);
          s1 += to_half(y, p1, 16, ck[1], lr[1] - mu);
          const float top = fmaxf(mx, mz);
          if (!__any_sync(0xffffffffu, !(top <= m_ref + kLazy))) {
            tmem_st32(sc, p0);
            tmem_st32(sc + 32, p1);
            l = fmaf(s0, ex2(-lr[0]), fmaf(s1, ex2(-lr[1]), l));
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[w]);
            continue;
          }
        }
        float top = -INFINITY;
        // (the passes' loops stay rolled: with both halves of the tile written out the three roles'
        // code no longer fits the instruction caches, and the product issue waits for its own)
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          tmem_ld32(sc + 64 * u, x);
          tmem_ld32(sc + 64 * u + 32, y);
          tmem_ld_wait();
          if (!full) {
            const uint32_t b0 = u ? km[2] : km[0], b1 = u ? km[3] : km[1];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              x[k] = (b0 >> k) & 1u ? x[k] : 0xff800000u;
              y[k] = (b1 >> k) & 1u ? y[k] : 0xff800000u;
            }
          }
          const float mx = fmaxf(max32(x), max32(y));
          if (mx != -INFINITY) top = fmaxf(top, fmaf(mx, u ? ck[1] : ck[0], u ? to[1] : to[0]));
        }
        const bool up = top > m_ref + kLazy || (m_ref == -INFINITY && top > -INFINITY);
        const bool scale_o = up && m_ref != -INFINITY;
        const float m_new = up ? ceilf(top) : m_ref;
        if (__any_sync(0xffffffffu, scale_o)) {
          // O of this warpgroup's earlier tiles: their PV finished before S of this one did
          const float al = scale_o ? ex2(m_ref - m_new) : 1.f;
          l *= al;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld32(oc + 32 * c, x);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * al);
            tmem_st32(oc + 32 * c, x);
          }
          tmem_st_wait();
        }
        m_ref = m_new;
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          tmem_ld32(sc + 64 * u, x);
          tmem_ld32(sc + 64 * u + 32, y);
          tmem_ld_wait();
          const float cu = u ? ck[1] : ck[0], lu = u ? lr[1] : lr[0], off = lu - mu;
          const uint32_t b0 = u ? km[2] : km[0], b1 = u ? km[3] : km[1];
          const uint32_t c0 = sc + (TERMS == 2 ? 64 : 32) * u, c1 = c0 + (TERMS == 2 ? 32 : 16);
          float sum;
          if (full)
            sum = emit<TERMS, true>(x, c0, cu, off, 0u) + emit<TERMS, true>(y, c1, cu, off, 0u);
          else if (r.tree)
            sum = emit<2, false>(x, sc + 64 * u, cu, off, b0) + emit<2, false>(y, sc + 64 * u + 32, cu, off, b1);
          else
            sum = emit<TERMS, false>(x, c0, cu, off, b0) + emit<TERMS, false>(y, c1, cu, off, b1);
          l = fmaf(sum, ex2(-lu), l);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[w]);
      }
      // ---- epilogue: partial rows (A: 128 dims of the own row; B: 64 dims of the merged row)
      ok = __all_sync(0xffffffffu, ok && wait_parity(&o_full, 0, a.err, ERR_O));
      tc_fence_after();
      s_m[w][rl] = m_ref;
      s_l[w][rl] = l;
      ok = bar_and(1, 256, ok);
      if (ok) {
        if (r.tree) (void)wait_parity(&w_full[0], 0, a.err, ERR_W);  // (long complete: orders s_q[0][0])
        const float unit = (r.tree ? s_q[0][0] : vref) * (1.f / (1 << PB));
        float M = m_ref, Lsum = l, fa = unit, fb = 0.f;
        const bool other = !two && items > 1;
        if (!two) {
          const float m0 = s_m[0][rl], m1 = s_m[1][rl];
          M = fmaxf(m0, m1);
          fa = m0 == -INFINITY ? 0.f : ex2(m0 - M);
          fb = m1 == -INFINITY ? 0.f : ex2(m1 - M);
          Lsum = fa * s_l[0][rl] + fb * s_l[1][rl];
          fa *= unit;
          fb *= unit;
        }
        const float back = kvq_settle(M, Lsum);
        fa *= back;
        fb *= back;
        // slices of 32 dims staged as 128-byte-swizzled rows over the Q area and both code
        // rings (every product has finished), then one TMA store each
        for (int c = two ? 0 : 2 * w; c < (two ? 4 : 2 * w + 2); ++c) {
          uint32_t x[32], y[32];
          tmem_ld32(lb + col_o(two ? w : 0) + 32 * c, x);
          if (other) tmem_ld32(lb + col_o(1) + 32 * c, y);
          tmem_ld_wait();
          uint8_t* dst = smem + ((two ? 4 * w : 0) + c) * T8 + rl * 128;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = __uint_as_float(x[4 * q + e]) * fa;
              if (other) f[e] = fmaf(__uint_as_float(y[4 * q + e]), fb, f[e]);
            }
            *reinterpret_cast<float4*>(dst + ((q ^ (rl & 7)) << 4)) = make_float4(f[0], f[1], f[2], f[3]);
          }
        }
        const size_t prow = (static_cast<size_t>(bh) * a.splits + piece) * a.rows_pad + row0;
        if (live && (two || w == 0))
          *reinterpret_cast<float2*>(a.part_ml + (prow + (two ? w * 128 : 0) + rl) * 2) = make_float2(M, Lsum);
        fence_proxy_async_smem();
        bar_sync(2 + (two ? w : 0), two ? 128 : 256);
        if (qd == 0 && lane == 0 && (two || w == 0)) {
          const int valid = RG - row0 - (two ? w * 128 : 0);  // boxes of 32 rows x 32 columns
          for (int g = 0; g < 128 && g < valid; g += 32)
            for (int c = 0; c < 4; ++c)
              tma_store_2d(&tm.po, smem + ((two ? 4 * w : 0) + c) * T8 + g * 128, 32 * c,
                           static_cast<int>(prow) + (two ? w * 128 : 0) + g);
          bulk_commit();
          if (a.coop)
            bulk_wait0();  // other CTAs of this launch read the rows
          else
            bulk_wait_read0();  // the combine kernel reads them once this grid has completed
          fence_proxy_async_global();
        }
      }
      if (a.coop) {
        // The group's merge: count this piece into its group (request, KV head, row block), wait
        // until every piece that has work has counted, then merge an even share of its rows from
        // L2, a warp per row.  A piece that gave up counts too: the others need not wait for it.
        const int need = kvq_pieces(a, n_pref);
        __threadfence();
        bar_sync(1, 256);
        if (threadIdx.x == 0) go = kvq_group_wait(a.cnt + 2 * (bh * (a.rows_pad / (a.wr * 128)) + rb), need, a.err, ERR_GROUP) ? 1 : 0;
        bar_sync(1, 256);
        if (threadIdx.x == 255) kvq_group_leave(a.cnt + 2 * (bh * (a.rows_pad / (a.wr * 128)) + rb), need);  // (no one waits for this)
        if (go) {
          const int n = min(two ? 256 : 128, RG - row0);
          const int hi = (piece + 1) * n / need;
#pragma unroll 1
          for (int k = piece * n / need + warp; k < hi; k += 8) {
            const size_t base = (static_cast<size_t>(bh) * a.splits) * a.rows_pad + row0 + k;
            const int nd = node_of(a, row0 + k);
            kvq_merge_row<128, 20>(a, base, need, (static_cast<size_t>(b) * a.R + nd) * a.Hq + h * a.G + (row0 + k - nd * a.G),
                                   lane);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 15) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

template <int TERMS>
cudaError_t launch_tc(const KvqAttnPlan& p, const Maps& tm, const KvqAttnArgs& a, cudaStream_t s) {
  auto kern = tree_attn_kvq_tc_kernel<TERMS>;
  constexpr int SMEM = Lay<TERMS>::SMEM;
  static unsigned long long configured = 0;  // shared memory opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    // the register split needs all of them at launch (it would wait for more for ever)
    if (e == cudaSuccess && fa.numRegs != 128) e = cudaErrorInvalidKernelImage;
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * p.Hkv * p.row_blocks, p.splits);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeCooperative;  // all CTAs resident, or the launch fails
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.coop ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kvq_attn_tc(const KvqAttnPlan& p, const KvqAttnArgs& a, cudaStream_t s) {
  Maps tm;
  const unsigned long long rows = static_cast<unsigned long long>(p.B) * p.Hkv * p.P;
  const unsigned long long prows = static_cast<unsigned long long>(p.B) * p.Hkv * p.splits * p.rows_pad;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!make_tmap_2d(&tm.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.k8, 128, rows, 128, KT, sw) ||
      !make_tmap_2d(&tm.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.v8, 128, rows, 128, KT, sw) ||
      !make_tmap_2d(&tm.po, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.part_o, 128, prows, 32, 32, sw))
    return cudaErrorInvalidValue;
  return p.terms2 ? launch_tc<2>(p, tm, a, s) : launch_tc<1>(p, tm, a, s);
}

}  // namespace eagle
