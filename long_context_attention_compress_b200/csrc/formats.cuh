// The 4-bit and 8-bit storage formats of cache rows (definitions in include/hca.h): MXFP4 (E2M1 elements, one
// power-of-two scale per 32 channels) and FP8 (E4M3 elements, one f32 scale per 64 channels).
#pragma once

#include <string.h>

#include "common.cuh"

namespace hca {

// ---- MXFP4 ---------------------------------------------------------------------
constexpr int kFp4Group = 32;

// E2M1 value of a 4-bit code (bit 3 sign, bits 1-2 exponent e with bias 1, bit 0
// mantissa m): e = 0 gives 0 or 0.5, else (1 + m/2) 2^(e-1); built as f32 bits.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const uint32_t mag = e ? (((126u + e) << 23) | (m << 22)) : (m ? 0x3F000000u : 0u);
  return __uint_as_float(mag | ((c & 8u) << 28));
}

// Eight E2M1 codes (word nibbles 0..7, element order) times 2^X -> eight bf16, packed in
// pairs (o[k] = element 2k | element 2k+1 << 16).  The magnitudes come from byte
// tables by byte permutes (bf16 bits of 0, 0.5, 1, 1.5, 2, 3, 4, 6: high bytes
// 00 3F 3F 3F 40 40 40 40, low bytes 00 00 80 C0 00 40 80 C0; __byte_perm reads only
// bits 0-2 of each of the four low selector nibbles, so the codes serve as selectors
// as they are, sign bit included).  The signs (bit 3 of each nibble) join the high
// bytes before the pairs are formed: byte k of (codes << 4) holds element 2k's sign in
// its bit 7 and byte k of the codes element 2k+1's, so one permute per four elements
// and a mask line them up with the high bytes of those elements.  2^X is applied by one
// bf16x2 multiply, exact while every nonzero product stays a normal bf16
// (|X| <= 125: 0.5 * 2^X .. 6 * 2^X); beyond that the values are formed in f32 (as
// exact) and rounded once.
__device__ __forceinline__ void e2m1x8_to_bf16(uint32_t w, int X, uint32_t* o) {
  constexpr uint32_t kHiLo = 0x3F3F3F00u, kHiHi = 0x40404040u, kLoLo = 0xC0800000u, kLoHi = 0xC0804000u;
  if (X >= -125 && X <= 125) {
    const uint32_t w4 = w << 4, wh = w >> 16;
    // high bytes of elements 0-3 and 4-7, signs included; low bytes likewise
    const uint32_t h0 = __byte_perm(kHiLo, kHiHi, w) | (__byte_perm(w4, w, 0x5140u) & 0x80808080u);
    const uint32_t h1 = __byte_perm(kHiLo, kHiHi, wh) | (__byte_perm(w4, w, 0x7362u) & 0x80808080u);
    const uint32_t l0 = __byte_perm(kLoLo, kLoHi, w), l1 = __byte_perm(kLoLo, kLoHi, wh);
    uint32_t p[4];
    p[0] = __byte_perm(l0, h0, 0x5140u);
    p[1] = __byte_perm(l0, h0, 0x7362u);
    p[2] = __byte_perm(l1, h1, 0x5140u);
    p[3] = __byte_perm(l1, h1, 0x7362u);
    const uint32_t sb = (uint32_t)(127 + X) << 7;  // bf16 bits of 2^X
    const uint32_t sbits = sb | (sb << 16);
    __nv_bfloat162 sc;
    memcpy(&sc, &sbits, 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      __nv_bfloat162 v;
      memcpy(&v, &p[k], 4);
      v = __hmul2(v, sc);
      memcpy(&o[k], &v, 4);
    }
    return;
  }
  const float scf = ldexpf(1.f, X);
#pragma unroll
  for (int j = 0; j < 8; j += 2)
    o[j >> 1] = pack_bf16x2(e2m1_value((w >> (4 * j)) & 15u) * scf, e2m1_value((w >> (4 * j + 4)) & 15u) * scf);
}

// Byte permute whose selector nibbles are below 8 (what __byte_perm would first mask them to).
__device__ __forceinline__ uint32_t prmt_raw(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
// The same byte tables in straight-line code for every scale byte below 255: the multiplication by 2^X is exact, or
// rounds to the bf16 subnormal or infinity that the value has (2^-127 itself is a subnormal factor, which it takes).
// 14 half-rate and 4 multiply instructions per 8 codes; the conversion instruction (E2M1 -> f16 -> f32, times 2^X,
// -> bf16) takes 24, and mixing the two to use both pipes was slower in the attention, which is bound by issue slots.
__device__ __forceinline__ uint32_t e8m0_bf16x2(uint32_t scale_byte) {  // 2^X twice, as bf16
  const uint32_t b = scale_byte ? scale_byte << 7 : 0x0040u;
  return b | (b << 16);
}
__device__ __forceinline__ uint4 e2m1x8_times(uint32_t x, uint32_t factor) {
  constexpr uint32_t kHiLo = 0x3F3F3F00u, kHiHi = 0x40404040u, kLoLo = 0xC0800000u, kLoHi = 0xC0804000u;
  const uint32_t x4 = x << 4, m = x & 0x77777777u, mh = m >> 16;
  const uint32_t h0 = prmt_raw(kHiLo, kHiHi, m) | (prmt_raw(x4, x, 0x5140u) & 0x80808080u);
  const uint32_t h1 = prmt_raw(kHiLo, kHiHi, mh) | (prmt_raw(x4, x, 0x7362u) & 0x80808080u);
  const uint32_t l0 = prmt_raw(kLoLo, kLoHi, m), l1 = prmt_raw(kLoLo, kLoHi, mh);
  uint32_t t[4] = {prmt_raw(l0, h0, 0x5140u), prmt_raw(l0, h0, 0x7362u), prmt_raw(l1, h1, 0x5140u),
                   prmt_raw(l1, h1, 0x7362u)};
#pragma unroll
  for (int k = 0; k < 4; ++k) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t[k]) : "r"(t[k]), "r"(factor));
  return make_uint4(t[0], t[1], t[2], t[3]);
}
// A whole MXFP4 block: 32 codes (16 bytes) -> 32 bf16 as four 16-byte words.
__device__ __forceinline__ void e2m1x32_to_bf16(const uint4& w, uint32_t scale_byte, uint4* o) {
  const uint32_t f = e8m0_bf16x2(scale_byte);
  o[0] = e2m1x8_times(w.x, f);
  o[1] = e2m1x8_times(w.y, f);
  o[2] = e2m1x8_times(w.z, f);
  o[3] = e2m1x8_times(w.w, f);
}

// Nearest E2M1 code of a (already scaled) value, ties to the even code, saturating.
__device__ __forceinline__ uint32_t e2m1_code(float y) {
  const float a = fabsf(y);
  const uint32_t m = a <= 0.25f ? 0u : a < 0.75f ? 1u : a <= 1.25f ? 2u : a < 1.75f ? 3u
                   : a <= 2.5f ? 4u : a < 3.5f ? 5u : a <= 5.0f ? 6u : 7u;
  return (y < 0.f && m != 0u) ? (m | 8u) : m;
}

// Shared exponent of a block: floor(log2 amax) - 2 in [-127, 127]; -127 for an all-zero block.
__device__ __forceinline__ int mx_exponent(float amax) {
  if (!(amax > 0.f)) return -127;
  const int X = ilogbf(amax) - 2;
  return X < -127 ? -127 : (X > 127 ? 127 : X);
}

// ---- FP8 -----------------------------------------------------------------------
constexpr int kFp8Group = 64;
constexpr double kE4m3Max = 448.0;

// E4M3 byte of q (f64; a NaN gives 0), ties to even, saturating; sign bit 7, exponent bits 3-6
// (bias 7, field 0 = subnormal with spacing 2^-9), mantissa bits 0-2.
__device__ __forceinline__ uint32_t e4m3_encode(double q) {
  const uint32_t sign = q < 0.0 ? 0x80u : 0u;
  const double a = fabs(q);
  if (a >= kE4m3Max) return sign | 0x7Eu;  // 1.75 * 2^8 = 448
  int e = -6;
  if (a > 0.0) {
    int ex;
    frexp(a, &ex);  // a = f * 2^ex, f in [0.5, 1): floor(log2 a) = ex - 1
    e = ex - 1 < -6 ? -6 : ex - 1;
  }
  const double qq = ldexp(a, 3 - e);  // a / 2^(e-3), exact
  double fl = floor(qq);
  const double frac = qq - fl;
  if (frac > 0.5 || (frac == 0.5 && fmod(fl, 2.0) == 1.0)) fl += 1.0;
  int m = (int)fl;  // value = m * 2^(e-3), m in [0, 16]
  if (m >= 16) {    // rounded up into the next binade
    m = 8;
    ++e;
  }
  if (m < 8) return sign | ((uint32_t)m & 7u);  // subnormal (e = -6): exponent field 0
  return sign | ((uint32_t)(e + 7) << 3) | (uint32_t)(m - 8);
}

__device__ __forceinline__ float e4m3_decode(uint32_t b) {
  const uint32_t ex = (b >> 3) & 15u, m = b & 7u;
  const float mag = ex ? __uint_as_float(((ex + 120u) << 23) | (m << 20)) : (float)m * 0.001953125f;  // m * 2^-9
  return (b & 0x80u) ? -mag : mag;
}

}  // namespace hca
