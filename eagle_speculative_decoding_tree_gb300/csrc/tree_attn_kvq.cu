// tree_attn_kvq.cu -- tree attention over the 8-bit KV cache.
//
// The operation of tree_attn.cu (EAGLE review, terms "tree attention"; lesson glossary "Tree
// attention") with the prefix keys and values held as e4m3 codes with one scale per 64 rows:
//     s = scale q (code ks)        prefix key        s = scale q k        tree key (bf16)
//     out = sum 2^(s log2e - m) (code vs or v) / sum 2^(s log2e - m)
//
// How the 8-bit operands meet the tensor cores.  A code is exact as a half, so the prefix
// products run in half precision inputs with fp32 accumulators and the scales stay outside:
//   - a query row is multiplied by a power of two that puts its largest element in
//     [2^14, 2^15): bf16 to half is then exact down to elements of 2^-31 of that one, and off by
//     2^-39 of it at most below;
//   - ks multiplies the scores of its block (fp32);
//   - vs / vref, vref the largest vs of the CTA's key range, goes into the exponent of P, so
//     one accumulator serves blocks of different scales; the row sum takes it out again.  (Where
//     the tree shares it, its V gets a scale as a cache block's would be.)
//     P <= 2^15 in half: 11 significant bits down to 2^-24 of the row's largest p, steps of 2^-34
//     of it below, or 2^4 times as much of the largest p vs where that is less (kvq_toward).
// The reference maximum is kept in log2 units and rounded up to an integer, so that with
// power-of-two scales every exponent offset is exact.
//
// head_dim 128 runs on the tcgen05 kernels (tree_attn_kvq_tc.cu, up to 32 rows a KV head
// tree_attn_kvq_few.cu); the kernel here serves head_dim 64, EAGLE_ENGINE_MMA_SYNC and groups of
// more than 4096 query heads.
//
// Kernel (the split-KV shape of tree_attn.cu).  One CTA per (row block, split, request x KV
// head), sixteen warps of 16 query rows each: 128-key tiles of codes stream through a TMA ring
// (128-byte swizzle, 64-byte for head_dim 64; one thread refills a stage once its warps are past
// it), and a warp takes 16-key steps of them: the codes go from shared memory to registers once
// and become mma.sync m16n8k16 half fragments there, which is cheaper than writing a half tile
// back when there are few rows.  That is the bytes-bound case (few rows: a decode or chain
// step); a step is a chain of some 2000 cycles, so it takes sixteen warps' steps to keep
// up with HBM.  The fragments' orders are free choices: a thread's 16 bytes of a key are 16 head
// dims of the contraction, Q is stored to match; keys within a step are permuted by exchanging
// bits 0 and 2 so that the swizzled reads fall in different banks.
// wr warps stand side by side along the rows, 16 / wr along the keys; their states merge in
// shared memory at the end.  Splits write fp32 partials; when the whole grid fits on the SMs
// (cooperative launch) they merge in the kernel, else in kvq_combine_kernel.
#include <algorithm>

#include "common.cuh"
#include "kvq.cuh"
#include "kvq_merge.cuh"
#include "launch.h"
#include "sm100.cuh"
#include "tmap.h"

namespace eagle {
namespace {

using namespace sm100;

constexpr int KT = 128;       // keys per tile
constexpr int MAX_ST = 6;     // ring stages: 6 up to 64 rows a CTA, 4 beyond (the query rows' space)
constexpr int CW = 16;        // warps
// A row's reference moves when its maximum grew by more than 2^kLazy, and P is stored as
// p 2^PB vs / vref <= 2^15: a half's smallest step then is 2^-34 of the largest p.  A larger kLazy saves
// rescales, which are rare already at 2^4, and costs that range.
constexpr float kLazy = 4.f;
constexpr int PB = 11;

enum : int { ERR_FULL = 1, ERR_EMPTY = 2, ERR_GROUP = 256 };

struct Maps {
  CUtensorMap k, v;
};

__device__ __forceinline__ int prefix_len(const KvqAttnArgs& a, int b) {
  const int L = a.seq_len[b];
  return L < 0 ? 0 : (L > a.P ? a.P : L);
}
__device__ __forceinline__ int tree_rows(const KvqAttnArgs& a, int b) {
  if (!a.n_nodes) return a.R;
  const int n = a.n_nodes[b];
  return n < 0 ? 0 : (n > a.R ? a.R : n);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A warp's 16 rows (thread rows g and g + 8): running state.
template <int D>
struct RowState {
  float o[D / 8][4];
  float m[2], l[2];
};

// Scores t (log2 units, masked -inf) of 16 keys: moves the references if they must (see kvq_toward),
// turns t into P = p 2^(ld + PB) (in place) and adds the row sums.
template <int D>
__device__ __forceinline__ void soften(RowState<D>& st, float (&t)[2][4], float ld) {
  const float lr = ld + PB, back = ex2(-lr), toward = kvq_toward(ld);
  float m_new[2];
  bool move = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float mx = fmaxf(fmaxf(t[0][2 * i], t[0][2 * i + 1]), fmaxf(t[1][2 * i], t[1][2 * i + 1]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) + toward;
    const bool up = mx > st.m[i] + kLazy || (st.m[i] == -INFINITY && mx > -INFINITY);
    m_new[i] = up ? ceilf(mx) : st.m[i];
    move |= up;
  }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float al = st.m[i] == -INFINITY ? 0.f : ex2(st.m[i] - m_new[i]);
      st.m[i] = m_new[i];
      st.l[i] *= al;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        st.o[j][2 * i] *= al;
        st.o[j][2 * i + 1] *= al;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float off = lr - (st.m[i] == -INFINITY ? 0.f : st.m[i]);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 2 * i; e < 2 * i + 2; ++e) {
        t[j][e] = ex2(t[j][e] + off);
        sum += t[j][e];
      }
    st.l[i] = fmaf(sum, back, st.l[i]);
  }
}

template <int D>
__host__ __device__ constexpr int q_stride() { return D * 2 + 8; }  // bytes; 2 words past a bank row per row

template <int D, bool TERMS2>
__global__ void __launch_bounds__(CW * 32, 1)
    tree_attn_kvq_kernel(const __grid_constant__ Maps tm, const KvqAttnArgs a) {
  constexpr int TILE = KT * D;  // bytes of one K or V tile
  constexpr int CH = D / 16;    // 16-byte chunks of a row of codes
  constexpr int KS = D / 16;    // k-steps of QK^T
  constexpr int VB = D / 8;     // head dims of a thread's V column
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nst = a.nst;
  uint8_t* sq = ring + nst * 2 * TILE;
  __shared__ uint64_t full[MAX_ST], empty[MAX_ST];
  __shared__ float s_qs[CW * 16], s_m[CW][16], s_l[CW][16], s_vr[CW];
  __shared__ uint32_t s_tv[CW];
  __shared__ int go;

  const int rb = blockIdx.x, split = blockIdx.y, bh = blockIdx.z;
  const int b = bh / a.Hkv, h = bh % a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int wr = a.wr, wk = CW / wr, rows_cta = wr * 16;

  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], min(CW, wr * 8));  // the warps with a step in a tile
    }
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  const int L = prefix_len(a, b), Rb = tree_rows(a, b);
  const int RG = Rb * a.G;
  const int n_pref = (L + KT - 1) / KT;
  const int tps = kvq_tps(a, n_pref);
  const int u0 = split * tps, u1 = min(n_pref + 1, u0 + tps);
  const int n_pt = max(0, min(u1, n_pref) - u0);
  const bool tree = u0 <= n_pref && u1 == n_pref + 1;
  if (u0 > n_pref || rb * rows_cta >= RG) return;  // nothing of this request here (the combine skips it)
  const int blk0 = u0 * (KT / kQB);
  const int n_blk = n_pt > 0 ? (min(L, (u0 + n_pt) * KT) + kQB - 1) / kQB - blk0 : 0;
  const int nblk_all = (a.P + kQB - 1) / kQB;
  const float* ks = a.ks + static_cast<size_t>(bh) * nblk_all + blk0;
  const float* vs = a.vs + static_cast<size_t>(bh) * nblk_all + blk0;
  __syncthreads();  // barriers initialised

  const uint64_t policy = policy_evict_first();
  auto load_tile = [&](int t) {
    const int s = t % nst, y = bh * a.P + (u0 + t) * KT;
    mbar_arrive_expect_tx(&full[s], 2 * TILE);
    tma_load_2d_hint(ring + s * 2 * TILE, &tm.k, 0, y, &full[s], policy);
    tma_load_2d_hint(ring + s * 2 * TILE + TILE, &tm.v, 0, y, &full[s], policy);
  };
  int issued = 0;  // thread 0: tiles whose loads have gone out; the first before anything else is read
  if (threadIdx.x == 0)
    for (; issued < min(n_pt, nst); ++issued) load_tile(issued);
  // vref: the largest V scale of the key range; the tree's is chosen as a cache block's (vt)
  float vm = 0.f;
  for (int i = threadIdx.x; i < n_blk; i += CW * 32) vm = fmaxf(vm, __ldg(vs + i));
  uint32_t tm_bits = 0;  // the largest finite magnitude of the tree's V, as float bits
  if (tree) {
    const uint4* tvg = reinterpret_cast<const uint4*>(a.tv + static_cast<size_t>(bh) * a.R * D);
    for (int i = threadIdx.x; i < Rb * (D / 8); i += CW * 32) {
      const uint4 x = __ldg(tvg + i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t p0 = (w[e] << 16) & 0x7fff0000u, p1 = w[e] & 0x7fff0000u;
        tm_bits = max(tm_bits, max(p0 < 0x7f800000u ? p0 : 0u, p1 < 0x7f800000u ? p1 : 0u));
      }
    }
  }
  vm = warp_max(vm);
  tm_bits = __reduce_max_sync(0xffffffffu, tm_bits);
  if (lane == 0) {
    s_vr[warp] = vm;
    s_tv[warp] = tm_bits;
  }

  // Q rows as scaled halves: row r, element e at r * stride + 2 e
  for (int r = warp; r < rows_cta; r += CW) {
    const int row = rb * rows_cta + r;
    float f[D / 32];
    float am = 0.f;
    if (row < RG) {
      const uint16_t* src =
          a.q + ((static_cast<size_t>(b) * a.R + row / a.G) * a.Hq + h * a.G + row % a.G) * D + lane * (D / 32);
#pragma unroll
      for (int e = 0; e < D / 32; e += 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(src + e);
        f[e] = __uint_as_float(w << 16);
        f[e + 1] = __uint_as_float(w & 0xffff0000u);
      }
#pragma unroll
      for (int e = 0; e < D / 32; ++e) am = fmaxf(am, fabsf(f[e]) <= 3.402823466e38f ? fabsf(f[e]) : 0.f);
    } else {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) f[e] = 0.f;
    }
    am = warp_max(am);
    // am = f 2^x: multiply by 2^(14 - x); x at least -100 keeps both powers normal
    const int x = am > 0.f ? max(static_cast<int>(__float_as_uint(am) >> 23) - 127, -100) : 14;
    const float mul = __uint_as_float(static_cast<uint32_t>(127 + 14 - x) << 23);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2)
      *reinterpret_cast<uint32_t*>(sq + r * q_stride<D>() + (lane * (D / 32) + e) * 2) =
          pack_half(f[e] * mul, f[e + 1] * mul);
    if (lane == 0) s_qs[r] = __uint_as_float(static_cast<uint32_t>(127 + x - 14) << 23);
  }
  __syncthreads();
  float vref = s_vr[0];
  uint32_t tv_max = s_tv[0];
#pragma unroll
  for (int w = 1; w < CW; ++w) {
    vref = fmaxf(vref, s_vr[w]);
    tv_max = max(tv_max, s_tv[w]);
  }
  const float vt = kvq_scale(__uint_as_float(tv_max));
  vref = kvq_vref(fmaxf(vref, vt));
  const float vinv = 1.f / vref;

  bool ok = true;
  const int wrow = warp % wr, wkey = warp / wr;
  const int r0 = wrow * 16;  // first row of the warp within the CTA
  RowState<D> st;
#pragma unroll
  for (int j = 0; j < D / 8; ++j) st.o[j][0] = st.o[j][1] = st.o[j][2] = st.o[j][3] = 0.f;
  st.m[0] = st.m[1] = -INFINITY;
  st.l[0] = st.l[1] = 0.f;
  float cr[2];  // row factors of the scores
#pragma unroll
  for (int i = 0; i < 2; ++i) cr[i] = a.scale_log2 * s_qs[r0 + g + 8 * i];

  // ---- prefix: of the piece's 16-key steps (8 to a tile) those with index wkey modulo wk
  const int gs = (g & 2) | ((g & 1) << 2) | (g >> 2);      // key of column g within 8: bits 0 and 2 exchanged
  const int cs = ((2 * c) & 2) | ((2 * c) >> 2);           // key of column 2 c; column 2 c + 1 is cs + 4
  const int swz = D == 128 ? gs : (gs >> 1) & 3;           // chunk swizzle of key gs (and gs + 8)
  const uint32_t qrow = smem_u32(sq) + static_cast<uint32_t>((r0 + g) * q_stride<D>() + 32 * c);
  float ks_n = 0.f, vs_n = 0.f;
  if (n_pt > 0) {
    const int kb = min(wkey * 16 / kQB, n_blk - 1);
    ks_n = __ldg(ks + kb);
    vs_n = __ldg(vs + kb);
  }
  for (int sx = wkey; sx < n_pt * 8 && ok;) {
    const int t = sx >> 3, s = t % nst;
    ok = __all_sync(0xffffffffu, wait_parity(&full[s], (t / nst) & 1, a.err, ERR_FULL));
    if (!ok) break;
    const int nv = min(KT, L - (u0 + t) * KT);
    const uint8_t* tk = ring + s * 2 * TILE;
    const uint8_t* tv = tk + TILE;
    for (; sx < 8 * t + 8; sx += wk) {
      const int step = sx & 7;
      const float ksb = ks_n, vsb = vs_n;
      {  // the next step's scales
        const int kb = min((sx + wk) * 16 / kQB, n_blk - 1);
        ks_n = __ldg(ks + kb);
        vs_n = __ldg(vs + kb);
      }
      const int nk = nv - step * 16;  // valid keys of the step
      if (nk <= 0) continue;
      float sc[2][4];
      uint32_t kw[2][KS];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t* kr = tk + (step * 16 + 8 * j + gs) * D;
#pragma unroll
        for (int i = 0; i < CH / 4; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(kr + (((c + 4 * i) ^ swz) << 4));
          kw[j][4 * i] = u.x, kw[j][4 * i + 1] = u.y, kw[j][4 * i + 2] = u.z, kw[j][4 * i + 3] = u.w;
        }
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t qa[4];
        const uint32_t at = qrow + (k >> 2) * 128 + (k & 3) * 8;
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(qa[0]), "=r"(qa[2]) : "r"(at));
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(qa[1]), "=r"(qa[3]) : "r"(at + 8 * q_stride<D>()));
#pragma unroll
        for (int j = 0; j < 2; ++j) mma_f16(sc[j], qa, kvq_half2(kw[j][k]), kvq_half2(kw[j][k] >> 16));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[j][e] *= cr[e >> 1] * ksb;
          if (nk < 16 && 8 * j + cs + 4 * (e & 1) >= nk) sc[j][e] = -INFINITY;
        }
      soften<D>(st, sc, kvq_ld(vsb, vinv));
      uint32_t pa[4], pl[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = sc[k >> 1][2 * (k & 1)], x1 = sc[k >> 1][2 * (k & 1) + 1];
        pa[k] = pack_half(x0, x1);
        if (TERMS2) {
          const float2 hi = unpack_half(pa[k]);
          pl[k] = pack_half(x0 - hi.x, x1 - hi.y);
        }
      }
      // V: this thread's column g is head dims VB g .. VB g + VB - 1; its keys are columns
      // 2 c, 2 c + 1 of both 8-key halves
      uint32_t vw[4][VB / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kk = (i >> 1) * 8 + cs + 4 * (i & 1);
        const int sw = D == 128 ? kk & 7 : (kk >> 1) & 3;
        const uint8_t* vr = tv + (step * 16 + kk) * D;
        if (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(vr + ((g ^ sw) << 4));
          vw[i][0] = u.x, vw[i][1] = u.y, vw[i][VB / 4 - 2] = u.z, vw[i][VB / 4 - 1] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(vr + (((g >> 1) ^ sw) << 4) + (g & 1) * 8);
          vw[i][0] = u.x, vw[i][1] = u.y;
        }
        if (nk < 16 && kk >= nk) {
#pragma unroll
          for (int q = 0; q < VB / 4; ++q) vw[i][q] = 0u;
        }
      }
#pragma unroll
      for (int q = 0; q < VB / 4; ++q) {
        uint32_t e[2][2];  // [key half][bytes 0 1 / 2 3 of word q], as (key, key + 1) pairs
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          e[hf][0] = __byte_perm(vw[2 * hf][q], vw[2 * hf + 1][q], 0x5140);
          e[hf][1] = __byte_perm(vw[2 * hf][q], vw[2 * hf + 1][q], 0x7362);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t b0 = kvq_half2(e[0][y >> 1] >> (16 * (y & 1)));
          const uint32_t b1 = kvq_half2(e[1][y >> 1] >> (16 * (y & 1)));
          mma_f16(st.o[4 * q + y], pa, b0, b1);
          if (TERMS2) mma_f16(st.o[4 * q + y], pl, b0, b1);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    // refill the stage of the last tile that this warp was past before: the others are too by now
    if (threadIdx.x == 0) {
      while (issued < n_pt && issued - nst < t) {
        if (!wait_parity(&empty[issued % nst], (issued / nst - 1) & 1, a.err, ERR_EMPTY)) {
          ok = false;
          break;
        }
        load_tile(issued++);
      }
    }
    ok = __all_sync(0xffffffffu, ok);
  }
  // no copy may still be landing when the ring is used for the merge or the CTA ends
  if (threadIdx.x == 0)
    for (int s = 0; s < nst && s < issued; ++s)
      (void)wait_parity(&full[s], ((issued - 1 - s) / nst) & 1, a.err, ERR_FULL);

  // ---- the tree's own K/V (bf16, straight from global memory): 16-key steps shared out in
  // the same way; P always as three bf16 terms
  if (tree && ok) {
    const uint16_t* kb = a.tk + static_cast<size_t>(bh) * a.R * D;
    const uint16_t* vb = a.tv + static_cast<size_t>(bh) * a.R * D;
    const uint16_t* qp[2];
    const uint64_t* mp[2];
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = rb * rows_cta + r0 + g + 8 * i;
      live[i] = row < RG;
      const int node = live[i] ? row / a.G : 0, hq = h * a.G + (live[i] ? row % a.G : 0);
      qp[i] = a.q + ((static_cast<size_t>(b) * a.R + node) * a.Hq + hq) * D + 16 * c;
      mp[i] = a.anc_mask + (static_cast<size_t>(b) * a.R + node) * a.W;
    }
    // V enters as v / vt (a power of two: exact in bf16 down to 2^-126 of the largest), at most 448
    // like a code: with V as it is P would have to hold 1 / vref, beyond fp32 for tiny scales.
    const float ld = kvq_ld(vt, vinv);
    const __nv_bfloat162 vti = __float2bfloat162_rn(kvq_inverse(vt));
    auto scaled = [&](uint2 u) {
      const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u.x), vti);
      const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u.y), vti);
      return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    };
    for (int step = wkey; step * 16 < Rb; step += wk) {
      float sc[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int key = step * 16 + 8 * j + g;
        const uint16_t* kr = kb + static_cast<size_t>(min(key, Rb - 1)) * D + 16 * c;
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint2 kw = *reinterpret_cast<const uint2*>(kr + (k >> 2) * 64 + (k & 3) * 4);
          const uint2 q0 = *reinterpret_cast<const uint2*>(qp[0] + (k >> 2) * 64 + (k & 3) * 4);
          const uint2 q1 = *reinterpret_cast<const uint2*>(qp[1] + (k >> 2) * 64 + (k & 3) * 4);
          const uint32_t qa[4] = {q0.x, q1.x, q0.y, q1.y};
          mma_bf16(sc[j], qa, kw.x, kw.y);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k0 = step * 16;
        const uint64_t word = live[i] ? mp[i][k0 >> 6] : 0ull;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = k0 + 8 * j + 2 * c + e;
            const bool on = key < Rb && ((word >> (key & 63)) & 1ull);
            sc[j][2 * i + e] = on ? sc[j][2 * i + e] * a.scale_log2 : -INFINITY;
          }
      }
      soften<D>(st, sc, ld);
      uint32_t pt[3][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x0 = sc[k >> 1][2 * (k & 1)], x1 = sc[k >> 1][2 * (k & 1) + 1];
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          pt[u][k] = pack_bf(x0, x1);
          x0 -= __uint_as_float(pt[u][k] << 16);
          x1 -= __uint_as_float(pt[u][k] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int q = 0; q < VB / 4; ++q) {  // 4 head dims at a time
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = step * 16 + (i >> 1) * 8 + 2 * c + (i & 1);
          w[i] = key < Rb ? scaled(*reinterpret_cast<const uint2*>(vb + static_cast<size_t>(key) * D + VB * g + 4 * q))
                          : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t sel = (y & 1) ? 0x7632 : 0x5410;
          const uint32_t b0 = __byte_perm(y < 2 ? w[0].x : w[0].y, y < 2 ? w[1].x : w[1].y, sel);
          const uint32_t b1 = __byte_perm(y < 2 ? w[2].x : w[2].y, y < 2 ? w[3].x : w[3].y, sel);
#pragma unroll
          for (int u = 0; u < 3; ++u) mma_bf16(st.o[4 * q + y], pt[u], b0, b1);
        }
      }
    }
  }

  // ---- merge the key warps of the CTA: the row's states meet in shared memory
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], 1);
    st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], 2);
    if (c == 0) {
      s_m[warp][g + 8 * i] = st.m[i];
      s_l[warp][g + 8 * i] = st.l[i];
    }
  }
  __syncthreads();  // the ring is free
  float* so = reinterpret_cast<float*>(ring) + static_cast<size_t>(warp) * (16 * D);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < VB; j += 4)  // chunk index XORed with the row: the quads' rows fall in different banks
        *reinterpret_cast<float4*>(so + (g + 8 * i) * D + ((((VB * (2 * c + e) + j) >> 2) ^ g) << 2)) =
            make_float4(st.o[j][2 * i + e], st.o[j + 1][2 * i + e], st.o[j + 2][2 * i + e], st.o[j + 3][2 * i + e]);
  __syncthreads();
  const float unit = vref * (1.f / (1 << PB));  // (not into 1 / lsum: for the smallest vref that has few bits)
  constexpr int QD = D / 4;  // threads of a row, 4 dims each
  for (int idx = threadIdx.x; idx < rows_cta * QD; idx += CW * 32) {
    const int r = idx / QD, q = idx % QD;
    const int row = rb * rows_cta + r;
    if (row >= RG) break;
    const int w0 = r / 16, rr = r % 16;
    float M = -INFINITY;
    for (int k = 0; k < wk; ++k) M = fmaxf(M, s_m[w0 + k * wr][rr]);
    float lsum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < wk; ++k) {
      const int w = w0 + k * wr;
      const float f = s_m[w][rr] == -INFINITY ? 0.f : ex2(s_m[w][rr] - M);
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(ring) +
                                                        static_cast<size_t>(w) * (16 * D) + rr * D + ((q ^ (rr & 7)) << 2));
      lsum = fmaf(f, s_l[w][rr], lsum);
      acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
    }
    const float back = kvq_settle(M, lsum);
    acc.x *= back, acc.y *= back, acc.z *= back, acc.w *= back;
    if (a.splits > 1) {
      const size_t prow = (static_cast<size_t>(bh) * a.splits + split) * a.rows_pad + row;
      *reinterpret_cast<float4*>(a.part_o + prow * D + 4 * q) =
          make_float4(acc.x * unit, acc.y * unit, acc.z * unit, acc.w * unit);
      if (q == 0) *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(M, lsum);
    } else {
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // a row whose mask leaves nothing: zeros, lse -inf
      acc = make_float4(acc.x * inv * unit, acc.y * inv * unit, acc.z * inv * unit, acc.w * inv * unit);
      const size_t orow = (static_cast<size_t>(b) * a.R + row / a.G) * a.Hq + h * a.G + row % a.G;
      if (a.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D + 4 * q) = acc;
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + 4 * q) =
            make_uint2(pack_bf(acc.x, acc.y), pack_bf(acc.z, acc.w));
      if (a.lse && q == 0) a.lse[orow] = (M + log2f(lsum)) * 0.69314718055994531f;
    }
  }
  if (a.coop) {
    // the group's merge (request, KV head, row block): an even share of its rows, a warp per row
    const int need = kvq_pieces(a, n_pref);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
      go = kvq_group_wait(a.cnt + 2 * (bh * gridDim.x + rb), need, a.err, ERR_GROUP) ? 1 : 0;
    __syncthreads();
    if (threadIdx.x == CW * 32 - 1) kvq_group_leave(a.cnt + 2 * (bh * gridDim.x + rb), need);  // (no one waits for this)
    if (go) {
      const int n = min(rows_cta, RG - rb * rows_cta), hi = (split + 1) * n / need;
      for (int k = split * n / need + warp; k < hi; k += CW) {
        const int row = rb * rows_cta + k;
        kvq_merge_row<D, 16>(a, static_cast<size_t>(bh) * a.splits * a.rows_pad + row, need,
                             (static_cast<size_t>(b) * a.R + row / a.G) * a.Hq + h * a.G + row % a.G, lane);
      }
    }
  }
}

// Merge the splits of every row, a warp per row.
template <int D>
__global__ void __launch_bounds__(128) kvq_combine_kernel(const KvqAttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = (blockIdx.x * 4 + warp) * 4, bh = blockIdx.y;
  const int b = bh / a.Hkv, h = bh % a.Hkv;
  const int m = min(tree_rows(a, b) * a.G - r0, 4);
  const int n = kvq_pieces(a, (prefix_len(a, b) + KT - 1) / KT);
  if (m <= 0) return;
  const size_t base = static_cast<size_t>(bh) * a.splits * a.rows_pad + r0;
  auto orow = [&](int k) {
    return (static_cast<size_t>(b) * a.R + (r0 + k) / a.G) * a.Hq + h * a.G + (r0 + k) % a.G;
  };
  if (n <= 4) {
    kvq_merge_rows<D, 4>(a, base, n, m, lane, orow);
  } else if (n <= 8) {
#pragma unroll 1
    for (int k = 0; k < m; k += 2)
      kvq_merge_rows<D, 2>(a, base + k, n, min(m - k, 2), lane, [&](int u) { return orow(k + u); });
  } else {
#pragma unroll 1
    for (int k = 0; k < m; ++k) kvq_merge_row<D, 16>(a, base + k, n, orow(k), lane);
  }
}

template <int D>
cudaError_t launch_combine(const KvqAttnPlan& p, const KvqAttnArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.R * p.G + 15) / 16, p.B * p.Hkv);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kvq_combine_kernel<D>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, bool T2>
cudaError_t launch_mma(const KvqAttnPlan& p, const Maps& tm, const KvqAttnArgs& a, cudaStream_t s) {
  auto kern = tree_attn_kvq_kernel<D, T2>;
  const int smem = 1024 + a.nst * 2 * KT * D + p.rows_per_cta * q_stride<D>();
  const int most = 1024 + std::max(4 * 2 * KT * D + CW * 16 * q_stride<D>(), MAX_ST * 2 * KT * D + 64 * q_stride<D>());
  // opt in to the largest size once per device (not a stream operation)
  static unsigned long long configured = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeCooperative;  // all CTAs resident, or the launch fails
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.coop ? 2 : 1;
  cfg.gridDim = dim3(p.row_blocks, p.splits, p.B * p.Hkv);
  cfg.blockDim = dim3(CW * 32);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, kern, tm, a);
  if (e != cudaSuccess || p.splits == 1 || p.coop) return e;
  return launch_combine<D>(p, a, s);
}

}  // namespace

// Prefix pieces of a request, beside its tree, on the tcgen05 kernels (one CTA per SM: they hold
// all of TMEM); base: groups (requests x KV heads x row blocks); a CTA costs about `extra` tiles'
// time besides its own (prologue, partials, meeting).  Either one wave of CTAs that shares every
// request's own length out evenly, so that a capacity far above the lengths in use leaves no CTA
// idle; or fixed pieces.  The lengths are not known here, so each choice is judged by two cases
// together: all requests of full length (waves of equal CTAs), and lengths spread evenly (the
// mean work, and a tail of most of a piece).  Measured: 8 requests of 1K to 16K x 8 heads 88 to
// 102 us with 3 to 8 pieces, 120 with 2, 210 with 1; 32 such 253 to 255 us with 3 or 4, 261 with 2,
// 276 with 6; 32 of 8K each 259 us with the 2 taken here, 238 with 1 (full lengths alone would
// choose 1; the two cases together do not); one of 8K 19.1 us in one wave.
// The plan's cost, in tiles' time, in *cost.
static long long choose_pieces(long long base, int tiles, int num_sms, int extra, bool* even, double* cost) {
  const long long one = std::min<long long>(num_sms / base - 1, tiles);
  *even = one >= 1;
  long long best = std::max<long long>(one, 1);
  double least = one >= 1 ? 2.0 * static_cast<double>((tiles + one - 1) / one + extra) : 1e30;
  for (int n = 1; n <= std::min(tiles, 64); ++n) {
    const int tps = (tiles + n - 1) / n;
    const double full = static_cast<double>((base * n + num_sms - 1) / num_sms) * (tps + extra);
    const double spread =
        static_cast<double>(base) / num_sms * (0.5 * tiles + extra * (0.5 * n + 1)) + 0.7 * (tps + extra);
    const double t = full + spread + extra;  // (and a second launch)
    if (t < least) {
      least = t;
      best = n;
      *even = false;
    }
  }
  *cost = least;
  return best;
}

void plan_kvq_attn(const eagle_attn_desc* d, int num_sms, KvqAttnPlan* p) {
  p->B = d->batch;
  p->R = d->rows;
  p->Hq = d->n_q_heads;
  p->Hkv = d->n_kv_heads;
  p->G = d->n_q_heads / d->n_kv_heads;
  p->D = d->head_dim;
  p->P = d->max_seq;
  p->W = (d->rows + 63) / 64;
  p->out_f32 = d->out_dtype == EAGLE_F32;
  p->terms2 = d->precision == EAGLE_ATTN_PRECISE;
  p->scale = d->scale;
  const int RG = p->R * p->G;
  const int tiles = (p->P + KT - 1) / KT;
  // head_dim 128 runs on tcgen05: up to 32 rows with the keys on the 128-row side, more in row
  // tiles of 128
  const bool tcgen = d->engine == EAGLE_ENGINE_AUTO && p->D == 128 && p->G <= 4096;
  p->few = tcgen && RG <= 32;
  p->tc = tcgen && !p->few;
  p->coop = p->even = false;
  if (p->tc || p->few) {
    const long long groups = static_cast<long long>(p->B) * p->Hkv, pairs = (RG + 255) / 256, blocks = (RG + 127) / 128;
    long long pieces = d->num_splits;
    double cost = 0.;
    p->wr = RG > 128 ? 2 : 1;
    if (pieces <= 0) pieces = choose_pieces(p->few ? groups : groups * (p->wr == 2 ? pairs : blocks), tiles, num_sms,
                                            p->few ? 10 : 6, &p->even, &cost);
    if (d->num_splits <= 0 && p->tc && p->wr == 2) {
      // Or a CTA for every 128 rows, with half as many pieces.  The codes are then read (from L2) and
      // widened twice, a row tile's 128 keys taking 1800 cycles instead of 1350, but a CTA has half
      // the query tile to stage and all of them together half the partials to exchange.  Measured
      // (8 KV heads, 61 nodes x 4): over 512 keys 14.7 against 19.6 us, 8K 19.0 against 20.7, 16K 26.8
      // against 28.8, 24K 35.0 against 34.3; 4 requests of 4K 32 against 39; 32 of 1K to 16K 277
      // against 270.
      bool even;
      double alone;
      const long long n = choose_pieces(groups * blocks, tiles, num_sms, 4, &even, &alone);
      if (0.65 * alone < cost) {
        p->wr = 1;
        pieces = n;
        p->even = even;
      }
    }
    p->rows_per_cta = p->few ? (RG <= 16 ? 16 : 32) : p->wr * 128;
    p->row_blocks = (RG + p->rows_per_cta - 1) / p->rows_per_cta;
    const long long base = groups * p->row_blocks;
    pieces = std::min<long long>(std::min<long long>(pieces, tiles), 255);
    p->tps = static_cast<int>((tiles + pieces - 1) / pieces);
    p->splits = (tiles + p->tps - 1) / p->tps + 1;
    p->coop = base * p->splits <= num_sms;
  } else {
    // rows of a CTA: as few warps along the rows as cover them, up to 16 x 16
    p->wr = 1;
    while (p->wr < CW && p->wr * 16 < RG) p->wr *= 2;
    p->rows_per_cta = p->wr * 16;
    p->row_blocks = (RG + p->rows_per_cta - 1) / p->rows_per_cta;
    // pieces of tps 128-key units (the tree counts as one): one wave of CTAs when the groups
    // are few, pieces of at least 16 units when they are many
    const long long base = static_cast<long long>(p->B) * p->Hkv * p->row_blocks;
    long long splits = d->num_splits > 0 ? d->num_splits : std::max<long long>(1, num_sms / base);
    if (d->num_splits <= 0 && p->B > 1) splits = std::max<long long>(splits, (tiles + 1) / 16);
    p->even = p->B == 1;
    splits = std::min<long long>(std::min<long long>(splits, tiles + 1), 256);
    p->tps = static_cast<int>((tiles + splits) / splits);
    p->splits = (tiles + p->tps) / p->tps;
    p->coop = p->splits > 1 && base * p->splits <= num_sms;
  }
  p->rows_pad = p->row_blocks * p->rows_per_cta;
  p->off_err = 0;
  size_t off = 256;
  p->off_cnt = off;
  // the meeting groups' counters, at most one group an SM: the same place whatever the descriptor,
  // so that the partials of one never lie where another expects its counters at zero
  off += (static_cast<size_t>(num_sms) * 8 + 255) / 256 * 256;
  p->off_o = p->off_ml = 0;
  if (p->splits > 1) {
    const size_t rows = static_cast<size_t>(p->B) * p->Hkv * p->splits * p->rows_pad;
    p->off_o = off;
    off += (rows * p->D * 4 + 255) / 256 * 256;
    p->off_ml = off;
    off += rows * 8;
  }
  p->total = off;
}

cudaError_t launch_kvq_attn(const KvqAttnPlan& p, const void* q, const void* k8, const float* ks, const void* v8,
                            const float* vs, const void* tree_k, const void* tree_v, const int32_t* seq_len,
                            const int32_t* n_nodes, const uint64_t* anc_mask, void* out, float* lse, void* ws,
                            cudaStream_t s) {
  KvqAttnArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k8 = static_cast<const uint8_t*>(k8);
  a.ks = ks;
  a.v8 = static_cast<const uint8_t*>(v8);
  a.vs = vs;
  a.tk = static_cast<const uint16_t*>(tree_k);
  a.tv = static_cast<const uint16_t*>(tree_v);
  a.seq_len = seq_len;
  a.n_nodes = n_nodes;
  a.anc_mask = anc_mask;
  a.out = out;
  a.lse = lse;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.part_o = reinterpret_cast<float*>(w + p.off_o);
  a.part_ml = reinterpret_cast<float*>(w + p.off_ml);
  a.err = reinterpret_cast<int*>(w + p.off_err);
  a.cnt = reinterpret_cast<int*>(w + p.off_cnt);
  a.coop = p.coop ? 1 : 0;
  a.even = p.even ? 1 : 0;
  a.B = p.B;
  a.R = p.R;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.G = p.G;
  a.P = p.P;
  a.W = p.W;
  a.splits = p.splits;
  a.tps = p.tps;
  a.rows_pad = p.rows_pad;
  a.out_f32 = p.out_f32;
  a.wr = p.wr;
  a.tc = p.tc || p.few ? 1 : 0;
  a.nst = p.rows_per_cta <= 64 ? MAX_ST : 4;
  a.g_inv = p.G > 1 ? static_cast<uint32_t>(((1ull << 32) + p.G - 1) / p.G) : 0u;
  a.scale = p.scale;
  a.scale_log2 = p.scale * kLog2e;
  if (p.tc || p.few) {
    const cudaError_t e = p.tc ? launch_kvq_attn_tc(p, a, s) : launch_kvq_attn_few(p, a, s);
    return e != cudaSuccess || p.coop ? e : launch_combine<128>(p, a, s);
  }
  Maps tm;
  const unsigned long long rows = static_cast<unsigned long long>(p.B) * p.Hkv * p.P;
  const CUtensorMapSwizzle sw = p.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!make_tmap_2d(&tm.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, k8, p.D, rows, p.D, KT, sw) ||
      !make_tmap_2d(&tm.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, v8, p.D, rows, p.D, KT, sw))
    return cudaErrorInvalidValue;
  if (p.D == 64) return p.terms2 ? launch_mma<64, true>(p, tm, a, s) : launch_mma<64, false>(p, tm, a, s);
  return p.terms2 ? launch_mma<128, true>(p, tm, a, s) : launch_mma<128, false>(p, tm, a, s);
}

}  // namespace eagle
