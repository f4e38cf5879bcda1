// kvq.cuh -- the 8-bit KV cache format shared by its kernels.
//
// A cache row holds e4m3 codes; the EAGLE_KVQ_BLOCK rows of an aligned block share one
// fp32 scale for each head, value = code * scale.  The writers choose the scale as the
// smallest power of two s with amax <= 448 s: dividing by it is exact, so a stored value
// is the nearest e4m3 value and nothing else is rounded, and a scale that grows later
// moves the codes already stored without rounding them again (below the new scale's
// normal range they lose the bits that e4m3's subnormals do not have).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace eagle {

constexpr int kQB = EAGLE_KVQ_BLOCK;

// Smallest power of two s >= 2^-126 with amax <= 448 s; 0 for amax == 0.  448 = 1.75 * 2^8:
// with amax = f 2^x, 1 <= f < 2, s = 2^(x - 8) if f <= 1.75, else 2^(x - 7).
__device__ __forceinline__ float kvq_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  const int x = static_cast<int>(u >> 23) - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);  // biased exponent of s
  return __uint_as_float(static_cast<uint32_t>(x < 1 ? 1 : x) << 23);
}

// 1 / s for a power-of-two scale (1 for the scale of a block of zeros).
__device__ __forceinline__ float kvq_inverse(float s) { return s > 0.f ? 1.f / s : 1.f; }

// The V scale that an accumulator's others refer to: the largest of its keys, at least the
// smallest normal number (its inverse is finite then).
__device__ __forceinline__ float kvq_vref(float largest) { return fmaxf(largest, 0x1p-126f); }

// log2 of a key's V scale against vref, what its P carries in the exponent.  At least -100, so that
// row sums of p = P 2^-ld stay in fp32: a smaller scale counts as 2^-100 vref.
__device__ __forceinline__ float kvq_ld(float vs, float vinv) { return fmaxf(__log2f(vs * vinv), -100.f); }

// A row's reference follows the largest score + kvq_toward(ld), not the largest score alone: P's
// largest is then within 2^4 of what weighs most in the sum of P V, however small its V scale is
// against the others of the piece, and P's fewer bits cut only what is small against that.  (With
// the largest score alone, keys with all the weight under a scale of 2^-32 vref came out with four
// bits or none.)  Scales within 2^4 of vref, as in ordinary caches, do not move it: following ld all
// the way made the references move more often there, 120 against 112 us for 61 nodes over 128K.
__device__ __forceinline__ float kvq_toward(float ld) { return fminf(ld + 4.f, 0.f); }

// A row sum far above its reference, as where the weight is under small V scales, brought below
// 2^18 by moving the reference (log2 units) up: the factor for what else refers to it.
__device__ __forceinline__ float kvq_settle(float& m, float& l) {
  const int e = max(static_cast<int>(__float_as_uint(l) >> 23) - (127 + 17), 0);
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  m += static_cast<float>(e);
  l *= f;
  return f;
}

// Two floats to e4m3 codes, nearest even, `lo` in the low byte.  A value that is not finite
// becomes the NaN code: it must not read back as an ordinary number.
__device__ __forceinline__ uint32_t kvq_code2(float lo, float hi) {
  const float nan = __uint_as_float(0x7fffffffu);
  lo = fabsf(lo) <= 3.402823466e38f ? lo : nan;
  hi = fabsf(hi) <= 3.402823466e38f ? hi : nan;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes (the low 16 bits of w) as packed halves; exact.
__device__ __forceinline__ uint32_t kvq_half2(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ float2 kvq_float2(uint32_t w) {
  const uint32_t h = kvq_half2(w);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A query row's elements as 8-bit terms of their own products with the codes, two halves to the
// upper bytes of two halves each.  A term is what is left so far, rounded to its format's significant
// bits, and what it leaves is exact in a half; an e5m2 code is a half's upper byte, an e4m3 code the
// bits 13 .. 7 and the sign of a half times 2^-8 (subnormals too).  Integer instructions (conversions
// to and from e4m3 for the two terms: 32 requests of 1K to 16K 262.7 against 261.6 us, 61 nodes over
// 2K 15.6 against 15.4).
//
// Two terms (EAGLE_ATTN_FAST; the row's largest element in (224, 448]): e4m3 holds four of bf16's
// eight bits, and rounding leaves a rest of at most eight units, which three bits hold: e5m2, down to
// steps of 2^-16; or, where the terms' products are columns of their own (APART), 2^4 times it as
// e4m3.  Exact down to elements of 2^-13 of the row's largest; below, the first term is off by 2^-10 at
// most, the second's steps in it are 2^-13: 2^-14, below 2^-21 of the row's largest.
template <bool APART>
__device__ __forceinline__ void kvq_split2(uint32_t h, uint32_t& hi, uint32_t& lo) {
  const auto as_half = [](uint32_t x) { return *reinterpret_cast<const __half2*>(&x); };
  const auto as_bits = [](__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); };
  const auto both = [](float x) { return __floats2half2_rn(x, x); };
  const uint32_t t = (as_bits(__hmul2(as_half(h), both(0x1p-8f))) + 0x00400040u) & 0xff80ff80u;
  const __half2 d = __hfma2(as_half(t), both(-256.f), as_half(h));
  hi = (t << 1) | (t & 0x80008000u);
  if (APART) {
    const uint32_t l = as_bits(__hmul2(d, both(0x1p-4f))) + 0x00400040u;
    lo = (l << 1) | (l & 0x80008000u);
  } else {
    lo = as_bits(d) + 0x00800080u;
  }
}
constexpr float kApart = 0x1p-4f;  // what the second term counts when APART

// Three terms (EAGLE_ATTN_PRECISE; the row's largest element in (28672, 57344]), all e5m2: exact down
// to elements of 2^-23 of the row's largest, below that off by 2^-17, less than 2^-31 of it.
__device__ __forceinline__ void kvq_split3(uint32_t h, uint32_t (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    t[i] = h + 0x00800080u;
    const uint32_t c = t[i] & 0xff00ff00u;
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&c));
    h = *reinterpret_cast<const uint32_t*>(&d);
  }
}
// The power of two that a row with the largest magnitude `am` is divided by for either.
__device__ __forceinline__ float kvq_qscale(uint32_t am, bool three) {
  return kvq_scale(fmaxf(__uint_as_float(min(am, 0x7f7f0000u)), 0x1p-100f)) * (three ? 0x1p-7f : 1.f);
}
// The codes of two such pairs.
__device__ __forceinline__ uint32_t kvq_pack(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }

// Four codes of one scale to the codes of a larger one: ratio = old scale / new scale.
__device__ __forceinline__ uint32_t kvq_move4(uint32_t w, float ratio) {
  const float2 a = kvq_float2(w), b = kvq_float2(w >> 16);
  return kvq_code2(a.x * ratio, a.y * ratio) | (kvq_code2(b.x * ratio, b.y * ratio) << 16);
}

}  // namespace eagle
