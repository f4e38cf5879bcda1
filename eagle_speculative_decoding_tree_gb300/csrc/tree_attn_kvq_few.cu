// tree_attn_kvq_few.cu -- tree attention over the 8-bit KV cache for few query rows (R G <= 32,
// head_dim 128: single tokens, chains) on the tcgen05 tensor cores, with keys on the 128-row side
// of the products; tree_attn_kvq.cu has the operation.
//
// Few rows against a long cache are bound by the cache's bytes, so nothing else may cost much:
//     S^T = K Q^T     M = 128 keys (K codes as they lie), N = the rows' terms
//     O^T = V^T P^T   M = 128 head dims (V codes as they lie, MN-major), N = the rows' P terms
// Both read a tile's codes once, straight from the TMA ring; no tile is converted.  All rounding
// is on the small side:
//   q  as in tree_attn_kvq_tc.cu: two terms keep bf16's bits down to elements of 2^-13 of the row's
//      largest, EAGLE_ATTN_PRECISE's three down to 2^-23;
//   p  2^PB vs / vref is rounded to a half (11 bits) and that half is written as four e5m2 terms
//      of three bits each, exactly down to steps of 2^-29 of the largest p (the rest after the
//      first term is multiplied by 8, past e5m2's smallest steps).  EAGLE_ATTN_PRECISE: two more
//      terms of what the half left (2^-17 of p).  A term is the upper byte of what is left of the
//      half, cut off, and rounded for the last of them and PRECISE's: integer instructions
//      (conversions to e5m2: 58.0 against 56.8 us for the chain of 8 over 128K).  The terms are
//      columns of their own; their scales meet in the epilogue, in fp32.
// A row's running maximum would need every key's score; instead the exponentials are taken
// against a reference that moves (a slow path through shared memory) when some score (a small V scale
// counted in: kvq_toward) is more than 2^kLazy above it, which a vote of the tile's threads finds out.
//
// One CTA per (piece, request x KV head):
//   softmax warpgroups, two for every 16 rows: a thread is one key of the tile (a TMEM lane) for
//                   its 16 rows; the two take alternate tiles and keep states of their own
//   a TMA producer warp: 128-key tiles of K and V codes, ST stages each
//   a warp that issues every tcgen05.mma: QK0 QK1 | QK2 PV0 | QK3 PV1 | ...
// (32 rows a thread instead of 16 take as many instructions, but at 2.5 warps a scheduler only
// every second cycle issued one: 61.7 us against 58.0 for a chain of 8 over 128K.)
// TMEM: S of four tiles (a column per row and term of Q, or per row), then O of the even and the odd
// tiles (a column per row and term of P).
// Measured (8 KV heads, 4 query heads each, graph replay): one token over 128K tokens 46 us (5.8
// TB/s, 86 % of a device copy's rate), over 8K 9.7; a chain of 8 over 128K, fp32 and precise, 56.5 us,
// 2 of them for Q's third term (the loop's waits and product issue take about as long a tile as HBM does).
// Piece 0 is the tree (at most 32 bf16 keys), computed in fp32 on the ordinary cores; the others
// are tps tiles of the prefix.  Pieces write fp32 partials, merged in the kernel when the grid
// fits on the SMs (cooperative launch), else by kvq_combine_kernel.
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
constexpr int T8 = KT * 128;  // a tile of codes, 16 KB
constexpr float kLazy = 4.f;  // as in tree_attn_kvq.cu
constexpr int PB = 11;

enum : int { ERR_K = 1, ERR_KE = 2, ERR_VE = 8, ERR_S = 32, ERR_P = 64, ERR_O = 128, ERR_GROUP = 256,
             ERR_Q = 512 };

struct Maps {
  CUtensorMap k, v;
};

template <int NR, int TERMS>
struct Few {
  static constexpr int SW = NR / 2;                 // softmax warps: NR / 16 x 2 warpgroups
  static constexpr int NT = SW * 32 + (NR == 32 ? 128 : 64);  // threads (setmaxnreg wants whole warpgroups)
  static constexpr int NP = NR * TERMS;             // O columns of a tile parity, bytes of a key's P
  static constexpr int QT = TERMS > 4 ? 3 : 2;      // terms of Q
  // Q's terms: columns of their own in S, or as many more products into the same ones.  The first for
  // 16 rows (one token over 128K: 45.6 us, the second 46.2), the second for 32 (a chain of 8 over 8K 13.0
  // us, the first 13.3; six terms of P leave TMEM no room for the first: 53.5, with two S buffers and a
  // wait for each of them 54.5).
  static constexpr bool ONE_S = NR == 32;
  static constexpr int NS = ONE_S ? NR : QT * NR;   // S columns of a tile
  static constexpr int ST = NR == 32 ? 5 : 6;       // ring stages
  static constexpr int SM_Q = 0;                    // the terms' rows of 128 codes
  static constexpr int SM_P = SM_Q + QT * NR * 128;     // two buffers, blocks of 32 columns x 128 keys
  static constexpr int P1 = 128 * NP;
  static constexpr int SM_K = SM_P + 2 * P1;
  static constexpr int SM_V = SM_K + ST * T8;
  static constexpr int SMEM = SM_V + ST * T8 + 1024;
  static_assert(P1 % 1024 == 0 && SM_P % 1024 == 0, "alignment of the rings");
  static_assert(SMEM <= 232448 - 4096 && 4 * NS + 2 * NP <= 512, "shared memory, TMEM columns");
};

// Descriptor with the 32-byte swizzle (MN-major P: rows of 32 columns, 8 keys every `sbo` bytes,
// 32 columns every `lbo`).
__device__ __forceinline__ uint64_t desc_sw32(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (6ull << 61);
}

// kind::f8f6f4, fp32 accumulator, M = 128; formats e4m3 0, e5m2 1; mn: both operands MN-major.
__host__ __device__ constexpr uint32_t idesc8(int bfmt, int mn, int n) {
  return (1u << 4) | (static_cast<uint32_t>(bfmt) << 10) | (static_cast<uint32_t>(mn) << 15) |
         (static_cast<uint32_t>(mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

// By one elected lane of a converged warp (see tree_attn_kvq_tc.cu).
__device__ __forceinline__ void mma8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(id), "r"(acc)
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
// An e5m2 code is a half's upper byte: two mantissa bits of ten.  Half a step of it, for two halves.
constexpr uint32_t kHalfStep = 0x00800080u;
__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t times8_half2(uint32_t a) {
  const __half2 d = __hmul2(*reinterpret_cast<const __half2*>(&a), __floats2half2_rn(8.f, 8.f));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint64_t twice(float x) { return f32x2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Floats as integers in the same order (NaN above everything).
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

// Piece 0: the tree's own keys, fp32.  A warp per row, a lane per key, then a lane per 4 head dims.
template <int NT>
__device__ void tree_piece(const KvqAttnArgs& a, uint8_t* smem, int b, int bh, int h, int Rb, size_t prow0) {
  constexpr int LD = 272;  // bytes of a row of 128 bf16: 16 past, so that 8 lanes' rows cover the banks
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* sk = smem;
  uint8_t* sv = smem + 32 * LD;
  const uint4* kg = reinterpret_cast<const uint4*>(a.tk + static_cast<size_t>(bh) * a.R * 128);
  const uint4* vg = reinterpret_cast<const uint4*>(a.tv + static_cast<size_t>(bh) * a.R * 128);
  for (int i = tid; i < Rb * 16; i += NT) {
    *reinterpret_cast<uint4*>(sk + (i >> 4) * LD + (i & 15) * 16) = __ldg(kg + i);
    *reinterpret_cast<uint4*>(sv + (i >> 4) * LD + (i & 15) * 16) = __ldg(vg + i);
  }
  __syncthreads();
  for (int row = warp; row < Rb * a.G; row += NT / 32) {
    const int node = row / a.G;
    const uint4* q = reinterpret_cast<const uint4*>(
        a.q + ((static_cast<size_t>(b) * a.R + node) * a.Hq + h * a.G + row % a.G) * 128);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
    for (int c = 0; c < 16; ++c) {
      const uint4 x = __ldg(q + c), y = *reinterpret_cast<const uint4*>(sk + min(lane, Rb - 1) * LD + c * 16);
      const uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0 = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(w[e] << 16), s0);
        s1 = fmaf(__uint_as_float(u[e] & 0xffff0000u), __uint_as_float(w[e] & 0xffff0000u), s1);
      }
    }
    const uint64_t word = a.anc_mask[(static_cast<size_t>(b) * a.R + node) * a.W];
    const float t = lane < Rb && ((word >> lane) & 1ull) ? (s0 + s1) * a.scale_log2 : -INFINITY;
    const float M = warp_max(t);
    const float p = t == -INFINITY ? 0.f : ex2(t - M), l = warp_sum(p);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < Rb; ++j) {
      const uint2 y = *reinterpret_cast<const uint2*>(sv + j * LD + lane * 8);
      const float pj = __shfl_sync(0xffffffffu, p, j);
      o[0] = fmaf(pj, __uint_as_float(y.x << 16), o[0]);
      o[1] = fmaf(pj, __uint_as_float(y.x & 0xffff0000u), o[1]);
      o[2] = fmaf(pj, __uint_as_float(y.y << 16), o[2]);
      o[3] = fmaf(pj, __uint_as_float(y.y & 0xffff0000u), o[3]);
    }
    *reinterpret_cast<float4*>(a.part_o + (prow0 + row) * 128 + lane * 4) = make_float4(o[0], o[1], o[2], o[3]);
    if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + (prow0 + row) * 2) = make_float2(M, l);
  }
}

template <int NR, int TERMS>
__global__ void __launch_bounds__(Few<NR, TERMS>::NT, 1)
    tree_attn_kvq_few_kernel(const __grid_constant__ Maps tm, const KvqAttnArgs a) {
  using F = Few<NR, TERMS>;
  constexpr int ST = F::ST, SW = F::SW, HALVES = NR / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[ST], k_empty[ST], v_empty[ST], s_full[4], p_full[2], p_empty[2], q_full, o_full;
  __shared__ uint32_t tmem_base;
  __shared__ int go;
  // by tile parity:
  __shared__ float s_m[2][NR];                 // the rows' reference maxima (-inf: none yet)
  __shared__ __align__(16) float s_c[NR];      // (both) score factors of the rows
  __shared__ __align__(16) float s_mu[2][NR];  // minus the reference, 0 for none
  __shared__ __align__(16) float s_al[2][NR];  // slow path: the rows' rescale
  __shared__ float s_red[2][4][NR];            // slow path, epilogue: the warps' maxima / sums

  int piece, bh, rb;  // dispatch order as in tree_attn_kvq_tc.cu
  kvq_place(a, 1, piece, bh, rb);
  const int b = bh / a.Hkv, h = bh % a.Hkv;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (warp == SW + 1) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 2);  // a tile's K and V (one wait for both: 56.8 -> 54.4 us for a chain of 8 over 128K)
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&s_full[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&p_full[s], HALVES * 128);
      mbar_init(&p_empty[s], 1);
    }
    mbar_init(&q_full, SW);
    mbar_init(&o_full, 1);
    fence_barrier_init();
  }
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();

  int L = a.seq_len[b];
  L = L < 0 ? 0 : (L > a.P ? a.P : L);
  const int Rb = a.n_nodes ? min(max(a.n_nodes[b], 0), a.R) : a.R;
  const int RG = Rb * a.G;
  const int n_pref = (L + KT - 1) / KT;
  const int tps = kvq_tps(a, n_pref);
  const int tile0 = (piece - 1) * tps;
  const int n = piece == 0 || RG == 0 ? 0 : max(0, min(tps, n_pref - tile0));
  const bool tree = piece == 0 && RG > 0, work = n > 0;
  const size_t prow0 = (static_cast<size_t>(bh) * a.splits + piece) * a.rows_pad;
  const uint32_t tb = tmem_base;
  auto col_s = [](int i) { return static_cast<uint32_t>((i & 3) * F::NS); };
  auto col_o = [](int w) { return static_cast<uint32_t>(4 * F::NS + w * F::NP); };

  // the group's merge (request, KV head): an even share of its rows, a warp per row
  const int need = kvq_pieces(a, n_pref);
  auto merge = [&](int warps) {
    if (!a.coop) return;
    __threadfence();
    bar_sync(5, warps * 32);
    if (threadIdx.x == 0) go = kvq_group_wait(a.cnt + 2 * bh, need, a.err, ERR_GROUP) ? 1 : 0;
    bar_sync(5, warps * 32);
    if (threadIdx.x == warps * 32 - 1) kvq_group_leave(a.cnt + 2 * bh, need);  // (no one waits for this)
    if (!go) return;
    const int hi = (piece + 1) * RG / need;
    for (int k = piece * RG / need + warp; k < hi; k += warps)
      kvq_merge_row<128, 20>(a, static_cast<size_t>(bh) * a.splits * a.rows_pad + k, need,
                             (static_cast<size_t>(b) * a.R + k / a.G) * a.Hq + h * a.G + k % a.G, lane);
  };

  if (tree) {
    tree_piece<F::NT>(a, smem, b, bh, h, Rb, prow0);
    merge(F::NT / 32);
  } else if (warp >= SW) {
    // registers: 96 a thread at launch with 640 threads (61440); softmax 104, the others 64
    // (512 x 104 + 128 x 64 = 61440).  With 320 threads there are enough as it is.
    if (HALVES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (!work) {
    } else if (warp == SW) {
      // ------------------------------------------------------------ TMA producer (lane 0)
      if (lane == 0) {
        const uint64_t policy = policy_evict_first();
        const int y0 = bh * a.P + tile0 * KT;
        auto load = [&](const CUtensorMap& m, int at, uint64_t* bar, int t) {
          mbar_arrive_expect_tx(bar, T8);
          tma_load_2d_hint(smem + at, &m, 0, y0 + t * KT, bar, policy);
        };
        int k_in = 0, v_in = 0;
        for (int t = 0; t < n; ++t) {
          const int s = t % ST;
          if (t >= ST && !wait_parity(&k_empty[s], (t / ST - 1) & 1, a.err, ERR_KE)) break;
          load(tm.k, F::SM_K + s * T8, &full[s], t);
          ++k_in;
          if (t >= ST && !wait_parity(&v_empty[s], (t / ST - 1) & 1, a.err, ERR_VE)) break;
          load(tm.v, F::SM_V + s * T8, &full[s], t);
          ++v_in;
          // the first tile first: with the whole ring's loads ahead of them the queries and scales
          // would arrive last, and nothing can start without them
          if (t == 0 && !wait_parity(&q_full, 0, a.err, ERR_Q)) break;
        }
        // no copy may still be landing when the CTA ends
        if (k_in > v_in) mbar_arrive(&full[v_in % ST]);  // (gave up between the two)
        for (int s = 0; s < ST && s < k_in; ++s) (void)wait_parity(&full[s], ((k_in - 1 - s) / ST) & 1, a.err, ERR_K);
      }
    } else if (warp == SW + 1) {
      // ------------------------------------------------------------ tcgen05.mma issue
      auto wait = [&](uint64_t* bar, int parity, int code) {
        return __all_sync(0xffffffffu, wait_parity(bar, parity, a.err, code)) != 0;
      };
      const uint32_t tu = __shfl_sync(0xffffffffu, tb, 0);
      const int items = __shfl_sync(0xffffffffu, n, 0);
      const uint64_t dq = smem_desc_sw128(smem_u32(smem + F::SM_Q), 16, 1024);
      const uint64_t dk = smem_desc_sw128(smem_u32(smem + F::SM_K), 16, 1024);
      const uint64_t dv = smem_desc_sw128(smem_u32(smem + F::SM_V), T8, 1024);
      const uint64_t dp = desc_sw32(smem_u32(smem + F::SM_P), 4096, 256);
      auto qk = [&](int i) {
        // into the S of tile i - 4, which the softmax has read: its P came before PV(i - 4)
        const int s = i % ST;
        if (!wait(&full[s], (i / ST) & 1, ERR_K)) return false;
        tc_fence_after();
#pragma unroll
        for (int term = 0; term < (F::ONE_S ? F::QT : 1); ++term)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)  // (two terms: e4m3 the first, or both in columns of their own)
            mma8(tu + col_s(i), dk + s * (T8 >> 4) + ks * 2, dq + term * (NR * 8) + ks * 2,
                 idesc8(F::QT == 3 || term ? 1 : 0, 0, F::NS), term + ks > 0);
        commit(&s_full[i & 3]);
        commit(&k_empty[s]);
        return true;
      };
      auto pv = [&](int i) {
        const int s = i % ST, w = i & 1;
        if (!wait(&p_full[w], (i >> 1) & 1, ERR_P)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)  // 32 keys: 4 KB of V, 1 KB of every block of P
          mma8(tu + col_o(w), dv + s * (T8 >> 4) + ks * 256, dp + w * (F::P1 >> 4) + ks * 64, idesc8(1, 1, F::NP),
               (i >= 2 || ks > 0) ? 1u : 0u);
        commit(&v_empty[s]);
        commit(&p_empty[w]);
        return true;
      };
      bool ok = wait(&q_full, 0, ERR_Q);
      ok = ok && qk(0) && (items < 2 || qk(1));
      // the scores of a warpgroup's next tile come under its exponentials
#pragma unroll 1
      for (int i = 0; i < items && ok; ++i) {
        if (i + 2 < items) ok = qk(i + 2);
        ok = ok && pv(i);
      }
      commit(&o_full);
    }
  } else {
    if (HALVES == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    if (work) {
      // ------------------------------------------------------------ softmax: a thread per key
      const int w = (warp >> 2) & 1, qd = warp & 3;      // tile parity, quarter of the keys
      const int vote = 1 + (warp >> 2), g0 = (warp >> 3) * 16;  // named barrier; the first of its rows
      const int key = qd * 32 + lane;  // of a tile; TMEM lane
      // Q: eight lanes a row, dims 8 c .. and 64 + 8 c ..
      const int row = threadIdx.x >> 3, c = threadIdx.x & 7;
      uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
      if (row < min(RG, NR)) {
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((static_cast<size_t>(b) * a.R + row / a.G) * a.Hq + h * a.G + row % a.G) * 128 + 8 * c);
        x0 = __ldg(src);
        x1 = __ldg(src + 8);
      }
      // vref: the largest V scale of the piece; the scales of this key's blocks
      const int nblk = (a.P + kQB - 1) / kQB, blk0 = tile0 * (KT / kQB);
      const int n_blk = (min(L, (tile0 + n) * KT) + kQB - 1) / kQB - blk0;
      const float* ks = a.ks + static_cast<size_t>(bh) * nblk + blk0;
      const float* vs = a.vs + static_cast<size_t>(bh) * nblk + blk0;
      float vref = 0.f;
#pragma unroll 4
      for (int i = lane; i < n_blk; i += 32) vref = fmaxf(vref, __ldg(vs + i));
      vref = kvq_vref(warp_max(vref));
      const float vinv = 1.f / vref;
      if (threadIdx.x < NR * 8) {
        const uint32_t u[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        uint32_t am = 0;  // the row's largest magnitude, as bf16 bits (ordered as integers)
#pragma unroll
        for (int k = 0; k < 8; ++k) am = max(am, max((u[k] << 16) & 0x7fff0000u, u[k] & 0x7fff0000u));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
        // a row with an element that is not finite gets NaN scores
        const float qs = kvq_qscale(am, F::QT == 3);
        const float mul = __uint_as_float((254u << 23) - __float_as_uint(qs));  // 1 / qs, a power of two
        if (c == 0)
          s_c[row] = am < 0x7f800000u ? a.scale_log2 * qs : __uint_as_float(0x7fffffffu);
        uint32_t tq[F::QT][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t t[2][3];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t v = u[2 * k + e];
            const uint32_t h = half2_bits(__uint_as_float(v << 16) * mul, __uint_as_float(v & 0xffff0000u) * mul);
            if (F::QT == 3)
              kvq_split3(h, t[e]);
            else
              kvq_split2<!F::ONE_S>(h, t[e][0], t[e][1]);
          }
#pragma unroll
          for (int i = 0; i < F::QT; ++i) tq[i][k] = kvq_pack(t[0][i], t[1][i]);
        }
        uint8_t* d1 = smem + F::SM_Q + row * 128 + (((c >> 1) ^ (row & 7)) << 4) + 8 * (c & 1);
        uint8_t* d2 = smem + F::SM_Q + row * 128 + ((((c >> 1) + 4) ^ (row & 7)) << 4) + 8 * (c & 1);
#pragma unroll
        for (int i = 0; i < F::QT; ++i) {
          *reinterpret_cast<uint2*>(d1 + i * NR * 128) = make_uint2(tq[i][0], tq[i][1]);
          *reinterpret_cast<uint2*>(d2 + i * NR * 128) = make_uint2(tq[i][2], tq[i][3]);
        }
        fence_proxy_async_smem();
      }
      if (threadIdx.x < 2 * NR) {
        s_m[threadIdx.x / NR][threadIdx.x % NR] = -INFINITY;
        s_mu[threadIdx.x / NR][threadIdx.x % NR] = 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
      float kn, vn;
      auto fetch = [&](int t) {
        const int kb = min(2 * t + (qd >> 1), n_blk - 1);
        kn = __ldg(ks + kb);
        vn = __ldg(vs + kb);
      };
      fetch(min(w, n - 1));
      bar_sync(5, SW * 32);  // s_c, s_m, s_mu

      const uint32_t lb = tb + (static_cast<uint32_t>(qd * 32) << 16);
      uint64_t l2[8];  // row sums, in pairs
#pragma unroll
      for (int r = 0; r < 8; ++r) l2[r] = 0ull;
      bool ok = true;
      for (int i = w; i < n; i += 2) {
        const float kc = kn, ld = kvq_ld(vn, vinv), lr = ld + PB;
        fetch(min(i + 2, n - 1));
        const uint64_t kc2 = twice(kc), lr2 = twice(lr);
        const int nv = min(KT, L - (tile0 + i) * KT);
        const bool on = key < nv;
        // A warp whose wait gave up goes on without waiting (the error word is set, nothing is
        // written): the others of its warpgroup may still count on it at the barriers below.
        ok = __all_sync(0xffffffffu, ok && wait_parity(&s_full[i & 3], (i >> 2) & 1, a.err, ERR_S));
        tc_fence_after();
        // x = score - reference (log2 units) of this key and every row
        float x[16];
        auto scores = [&]() {
          uint32_t hi[16], lo[16], third[16];
          tmem_ld16(lb + col_s(i) + g0, hi);
          if (!F::ONE_S) tmem_ld16(lb + col_s(i) + NR + g0, lo);
          if (!F::ONE_S && F::QT == 3) tmem_ld16(lb + col_s(i) + 2 * NR + g0, third);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < 16; r += 2) {
            const uint64_t c = *reinterpret_cast<const uint64_t*>(&s_c[g0 + r]);
            const uint64_t mu = *reinterpret_cast<const uint64_t*>(&s_mu[w][g0 + r]);
            uint64_t sum = f32x2(hi[r], hi[r + 1]);
            if (!F::ONE_S && F::QT == 2) sum = fma_f32x2(f32x2(lo[r], lo[r + 1]), twice(kApart), sum);
            if (!F::ONE_S && F::QT == 3)
              sum = add_f32x2(add_f32x2(sum, f32x2(lo[r], lo[r + 1])), f32x2(third[r], third[r + 1]));
            f32x2_split(fma_f32x2(sum, mul_f32x2(c, kc2), mu), x[r], x[r + 1]);
          }
          if (nv < KT) {
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = on ? x[r] : -INFINITY;
          }
        };
        scores();
        float over = i < 2 ? INFINITY : -INFINITY;  // (no reference yet)
#pragma unroll
        for (int r = 0; r < 16; r += 2) over = max3(over, x[r], x[r + 1]);
        // (a NaN score does not raise `over`: it spoils its row whatever the reference)
        const bool fits = bar_and(vote, 128, over + kvq_toward(ld) <= kLazy);
        // P's buffer and O: free once the product of this parity's tile before has finished
        ok = __all_sync(0xffffffffu, ok && (i < 2 || wait_parity(&p_empty[w], ((i >> 1) - 1) & 1, a.err, ERR_P)));
        if (!fits) {
          int mine = 0;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int m = __reduce_max_sync(0xffffffffu, ordered(x[r] == x[r] ? x[r] + kvq_toward(ld) : -INFINITY));
            if (lane == r) mine = m;
          }
          if (lane < 16) s_red[w][qd][g0 + lane] = unordered(mine);
          bar_sync(vote, 128);
          if (key < 16) {
            const int r = g0 + key;
            const float old = s_m[w][r];
            const float top = fmaxf(fmaxf(s_red[w][0][r], s_red[w][1][r]), fmaxf(s_red[w][2][r], s_red[w][3][r])) - s_mu[w][r];
            const bool up = top > old + kLazy || (old == -INFINITY && top > -INFINITY);
            s_al[w][r] = !up || old == -INFINITY ? 1.f : ex2(old - ceilf(top));  // (no reference yet: all zero)
            if (up) {
              s_m[w][r] = ceilf(top);
              s_mu[w][r] = -ceilf(top);
            }
          }
          bar_sync(vote, 128);
#pragma unroll
          for (int r = 0; r < 8; ++r)
            l2[r] = mul_f32x2(l2[r], *reinterpret_cast<const uint64_t*>(&s_al[w][g0 + 2 * r]));
          if (i >= 2) {
            tc_fence_after();
#pragma unroll 1
            for (int u = 0; u < TERMS; ++u) {
              uint32_t o[16];
              tmem_ld16(lb + col_o(w) + u * NR + g0, o);
              tmem_ld_wait();
#pragma unroll
              for (int r = 0; r < 16; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * s_al[w][g0 + r]);
              tmem_st16(lb + col_o(w) + u * NR + g0, o);
            }
            tmem_st_wait();
          }
          scores();  // against the new reference
        }
        // P: 16 bytes of every term
        const uint64_t back2 = twice(ex2(-lr));
        uint32_t hh[8], ll[8];
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          float y0, y1;
          f32x2_split(add_f32x2(f32x2(__float_as_uint(x[r]), __float_as_uint(x[r + 1])), lr2), y0, y1);
          const float p0 = ex2(y0), p1 = ex2(y1);
          const uint64_t p2 = f32x2(__float_as_uint(p0), __float_as_uint(p1));
          l2[r >> 1] = fma_f32x2(p2, back2, l2[r >> 1]);
          hh[r >> 1] = half2_bits(p0, p1);
          if (TERMS > 4) {
            // what the half left, by 2^11: a half's last place against its first
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh[r >> 1]));
            f32x2_split(mul_f32x2(add_f32x2(p2, f32x2(__float_as_uint(-f.x), __float_as_uint(-f.y))), twice(2048.f)), y0,
                        y1);
            ll[r >> 1] = half2_bits(y0, y1);
          }
        }
        uint8_t* pb = smem + F::SM_P + w * F::P1 + key * 32;
        const int flip = ((key >> 2) & 1) << 4;
#pragma unroll
        for (int u = 0; u < TERMS; ++u) {
          uint32_t c4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t &y0 = u < 4 ? hh[2 * k] : ll[2 * k], &y1 = u < 4 ? hh[2 * k + 1] : ll[2 * k + 1];
            const uint32_t t0 = u < 3 ? y0 : y0 + kHalfStep, t1 = u < 3 ? y1 : y1 + kHalfStep;
            c4[k] = __byte_perm(t0, t1, 0x7531);  // the upper bytes
            if (u != 3 && u != TERMS - 1) {       // exact: what a term leaves of a half
              y0 = sub_half2(y0, t0 & 0xff00ff00u);
              y1 = sub_half2(y1, t1 & 0xff00ff00u);
              if (u == 0) {
                y0 = times8_half2(y0);
                y1 = times8_half2(y1);
              }
            }
          }
          const int col = u * NR + g0;  // first of 16 columns: block col / 32, 16-byte half (col / 16) % 2
          *reinterpret_cast<uint4*>(pb + (col >> 5) * 4096 + ((col & 16) ^ flip)) = make_uint4(c4[0], c4[1], c4[2], c4[3]);
        }
        if (!on) {
          // V rows behind the prefix: zeros, whatever they hold (their P is 0)
          ok = ok && wait_parity(&full[i % ST], (i / ST) & 1, a.err, ERR_K);
          uint4* v = reinterpret_cast<uint4*>(smem + F::SM_V + (i % ST) * T8 + key * 128);
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&p_full[w]);
        ok = __all_sync(0xffffffffu, ok);
      }
      // ---- epilogue: the parities' states meet; a thread is now one head dim for its 16 rows
      // (the row sums while the last product runs)
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        float y0, y1;
        f32x2_split(l2[r >> 1], y0, y1);
        y0 = warp_sum(y0);
        y1 = warp_sum(y1);
        if (lane == 0) {
          s_red[w][qd][g0 + r] = y0;
          s_red[w][qd][g0 + r + 1] = y1;
        }
      }
      bool done = __all_sync(0xffffffffu, ok && wait_parity(&o_full, 0, a.err, ERR_O));
      tc_fence_after();
      done = bar_and(5, SW * 32, done);
      if (done) {
        const float unit = vref * (1.f / (1 << PB));
        const bool two = n > 1;
        float* so = reinterpret_cast<float*>(smem + F::SM_K);  // [NR][128]: the ring is free
        float o[16];
        if (w == 0 || two) {
          uint32_t y[16];
#pragma unroll
          for (int u = 0; u < TERMS; ++u) {
            tmem_ld16(lb + col_o(w) + u * NR + g0, y);
            tmem_ld_wait();
            const float f = unit * (u == 0 ? 1.f : (u < 4 ? 0.125f : 1.f / 2048.f));
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] = u == 0 ? __uint_as_float(y[r]) * f : fmaf(__uint_as_float(y[r]), f, o[r]);
          }
        }
        if (w == 1 && two) {
#pragma unroll
          for (int r = 0; r < 16; ++r) so[(g0 + r) * 128 + key] = o[r];
        }
        if (w == 0 && key < 16) {  // a row's weights of the two parities, its maximum and sum
          const int r = g0 + key;
          const float m0 = s_m[0][r], m1 = two ? s_m[1][r] : -INFINITY;
          float M = fmaxf(m0, m1);
          const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
          const float l0 = (s_red[0][0][r] + s_red[0][1][r]) + (s_red[0][2][r] + s_red[0][3][r]);
          const float l1 = (s_red[1][0][r] + s_red[1][1][r]) + (s_red[1][2][r] + s_red[1][3][r]);
          float l = fmaf(f0, l0, f1 * l1);
          const float back = kvq_settle(M, l);
          s_al[0][r] = f0 * back;
          s_al[1][r] = f1 * back;
          if (r < RG) *reinterpret_cast<float2*>(a.part_ml + (prow0 + r) * 2) = make_float2(M, l);
        }
        bar_sync(5, SW * 32);
        if (w == 0) {
          float* po = a.part_o + (prow0 + g0) * 128 + key;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            if (g0 + r >= RG) break;
            float y = o[r] * s_al[0][g0 + r];
            if (two) y = fmaf(so[(g0 + r) * 128 + key], s_al[1][g0 + r], y);
            po[r * 128] = y;
          }
        }
      }
      merge(SW);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == SW + 1) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

template <int NR, int TERMS>
cudaError_t launch_few(const KvqAttnPlan& p, const Maps& tm, const KvqAttnArgs& a, cudaStream_t s) {
  auto kern = tree_attn_kvq_few_kernel<NR, TERMS>;
  constexpr int smem = Few<NR, TERMS>::SMEM;
  static unsigned long long configured = 0;  // shared memory opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    // the register split needs all of them at launch (it would wait for more for ever)
    if (e == cudaSuccess && NR == 32 && fa.numRegs != 96) e = cudaErrorInvalidKernelImage;
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * p.Hkv, p.splits);
  cfg.blockDim = dim3(Few<NR, TERMS>::NT);
  cfg.dynamicSmemBytes = smem;
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

cudaError_t launch_kvq_attn_few(const KvqAttnPlan& p, const KvqAttnArgs& a, cudaStream_t s) {
  Maps tm;
  const unsigned long long rows = static_cast<unsigned long long>(p.B) * p.Hkv * p.P;
  if (!make_tmap_2d(&tm.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.k8, 128, rows, 128, KT, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tm.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.v8, 128, rows, 128, KT, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (p.rows_per_cta == 16) return p.terms2 ? launch_few<16, 6>(p, tm, a, s) : launch_few<16, 4>(p, tm, a, s);
  return p.terms2 ? launch_few<32, 6>(p, tm, a, s) : launch_few<32, 4>(p, tm, a, s);
}

}  // namespace eagle
