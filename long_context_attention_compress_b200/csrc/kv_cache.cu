// Rows into and out of a KV cache held in bf16, FP8 or FP4, flat, paged or a ring (sm_100a).
//
// kv_append_kernel.  y = x, or bf16(R_pos(x / sqrt(mean(x^2) + eps) * gamma)) with pos = (entry + 1)*rate - 1 and R
// the rotation of the last rope_dims channels; then y in the cache's form:
//   bf16; FP8: scale = f32(amax / 448) per 64 channels, the E4M3 value nearest to y / scale; FP4: 2^X per 32
//   channels, X = floor(log2 amax) - 2, the E2M1 value nearest to y * 2^-X; the last rope_dims channels bf16.
// One warp owns a row: lane l holds the 8-channel chunks l and l + 32, so a group's maximum is two (FP4) or three
// (FP8) shuffles away and nothing passes through memory between the input and the stored row; rows of at most 128
// channels that are only converted take half a warp.  The next row's load is always under way.
// Roundings.  With normalisation or rotation y is rounded to bf16 first (what the bf16 cache holds), as from the
// float64 value (by way of f32): a quantised code must not depend on which side of a midpoint an f32 normalisation falls.  Sum of
// squares and rotation are f64; the other channels are formed in f32, 8 ulps too low and too high (f32 is within 4),
// and redone in f64 only where the two round apart, or where a factor or a product may leave f32's normal range.  The codes are those of the stored-form definitions bit for bit:
// FP4 scaling is exact and the conversion rounds to nearest even; an f32 quotient (by the reciprocal, within 2 ulps)
// that is within 4 ulps of an E4M3 midpoint, or in E4M3's subnormal range, is decided on the f64 quotient.
// The angle is formed in turns from theta / 2 pi in two f64 words (a table made on the host) with an error-free product,
// so that its fraction is good to 2^-52 at any position and the sine and cosine need no long reduction.
// Bound: rows converted as they are, by the chain request, first entry, block table, store and by issue slots (24,577 FP4
// rows of 128 channels 5.3 us, 1.2 us of HBM time, 55 % of the slots taken); with normalisation and rotation by issue slots, 740 instructions a row at 0.6 a cycle and scheduler.  Measured, c = 512: 16,384 f32 rows
// normalised to FP4 19.3 us (6.0 us of HBM time; 7.5 us for the loads alone), 3,001 to FP8 in 13 ragged requests 7.4 us
// and 4,100 bf16 rows 6.5 us (a row or two a warp), 256 bf16 rows into rings 2.1 us, 8 rows 4.0 us: a row's chain of
// loads, f64 sum, inverse root and sine.  An f32 normalisation with error bounds and f64 behind it for every fifth row
// took 2 us longer for the 16,384.
//
// kv_gather_kernel.  The bf16 values of rows.  Each row is a chain of dependent loads (index, block table, row): a block
// resolves 16 rows at a time, one a thread, while its warps move the 16 before, two rows in flight per warp (their
// loads predicated, not branched around, so that they issue together); rows of at most 128 channels take half a warp,
// four in flight (24,577 rows of 128 FP4 channels 4.0 us, a warp a row 6.3).  bf16 rows move at the copy rate (8 x 8,191
// in 20.2 us); rows that are widened are bound by issue slots (two thirds of them taken, the ALU at 62 %, DRAM at 1.6 TB/s
// while the output stays in L2): 8 x 8,191 FP4 rows 18.5 us (13.9 at the copy rate), 32 x 1,024 selected FP8 rows 10.6 us
// (8.2); with four rows a warp and three blocks an SM 18.9 and 10.7, with two and six 18.5 and 11.4.

#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "formats.cuh"
#include "internal.h"

namespace hca {

__device__ unsigned int g_kv_append_error = 0;

namespace {
constexpr int kKvWarps = 4;        // warps per block
constexpr int kKvChunks = 2;       // 8-channel chunks per lane (c <= 512)
constexpr int kKvMaxPairs = 128;   // rope_dims <= 256

template <bool F32>
__device__ __forceinline__ void load8(const void* x, long long off, float* v) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + off);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(x) + off), v);
  }
}

// Eight E2M1 codes (element order, low nibble first) of values already scaled by 2^-X: nearest, ties to the even
// code, saturating; a negative value that rounds to zero has code 0.
__device__ __forceinline__ uint32_t e2m1x8_encode(const float* y) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  const uint32_t mag = (w | (w >> 1) | (w >> 2)) & 0x11111111u;  // bit 0 of each nibble: magnitude not zero
  return w & (0x77777777u | (mag << 3));
}

// Eight E4M3 codes of y / sc (see the head of this file).  The f64 decision is rare and long: one call outside the
// straight line, for the elements that need it.
__device__ __forceinline__ bool e4m3_doubtful(float q) {
  const int low = (int)(__float_as_uint(q) & 0xfffffu) - 0x80000;
  return fabsf(q) < 0.015625f || (low >= -4 && low <= 4);  // (a NaN is converted to the code of NaN)
}
// Rounded in f64 to a multiple of E4M3's spacing at its magnitude, ties to even, by adding and taking off 2^52 of them;
// what is left is a code's value (or past the largest one).
__device__ __noinline__ uint32_t e4m3_decide(float y, float sc) {
  if (y == 0.f) return 0u;  // (also of a group so small that its scale is 0)
  const double q = (double)y / (double)sc, a = fabs(q);
  const int e = max((__double2hiint(a) >> 20) - 1023, -6);
  const double big = __hiloint2double((e - 3 + 52 + 1023) << 20, 0);
  const float r = (float)copysign((a + big) - big, q);
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(h) : "f"(r));
  return r != 0.f ? h & 255u : q < 0.0 ? 128u : 0u;
}
__device__ __forceinline__ uint2 e4m3x8_encode(const float* y, float sc) {
  uint32_t w[4];
  uint32_t doubt = sc < 0x1p-100f ? 255u : 0u;  // (whose reciprocal may overflow)
  const float r_sc = 1.f / sc;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float q0 = y[2 * t] * r_sc, q1 = y[2 * t + 1] * r_sc;  // within 2 ulps of the quotient
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(q1), "f"(q0));
    w[t] = h;
    doubt |= (e4m3_doubtful(q0) ? 1u << (2 * t) : 0u) | (e4m3_doubtful(q1) ? 2u << (2 * t) : 0u);
  }
  uint2 r = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  while (doubt) {
    const int t = __ffs(doubt) - 1;
    doubt &= doubt - 1;
    float v = y[0];
#pragma unroll
    for (int u = 1; u < 8; ++u) v = t == u ? y[u] : v;
    const uint32_t c = e4m3_decide(v, sc), sh = 8 * (t & 3);
    if (t < 4) r.x = (r.x & ~(255u << sh)) | (c << sh);
    else r.y = (r.y & ~(255u << sh)) | (c << sh);
  }
  return r;
}

// Two f32 products in one instruction (16,384 normalised rows 0.6 us faster).
__device__ __forceinline__ float2 mul2(float a0, float a1, float b0, float b1) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
  return r;
}

// theta_j / 2 pi = base^(-2j / rope_dims) / 2 pi of each pair, as the sum of two doubles.
struct Turns {
  double hi[kKvMaxPairs], lo[kKvMaxPairs];
};
struct NoTurns {};  // (a launch that only converts does not carry the table)
template <bool XF>
using TurnsOf = std::conditional_t<XF, Turns, NoTurns>;

// Resident blocks per SM that the registers are held to.  Normalised, bf16 form: 7 against 6 took 6.4 against 6.8 us for
// 4,100 rows; FP8 and FP4, which need a few registers more: 6 against 7 took 24.9 against 25.3 us for 16,384 FP4 rows and
// their read-back.
constexpr int append_blocks(int form, bool xf) {
  return xf ? (form == HCA_KV_BF16 ? 7 : 6) : form == HCA_KV_FP8 ? 8 : 10;
}

// XF: with normalisation or rotation; without, a row is only converted.  LANES lanes a row: 16 for rows of at most 128
// channels that are only converted (the indexer's keys), else 32.
template <bool F32, int FORM, bool XF, int LANES>
__global__ void __launch_bounds__(32 * kKvWarps, append_blocks(FORM, XF))
    kv_append_kernel(KvAppend a, KvCache k, int base_rows, int one_more, const __grid_constant__ TurnsOf<XF> turns) {
  constexpr int kU = LANES == 32 ? kKvChunks : 1;  // chunks per lane
  __shared__ double2 s_turn[XF ? kKvMaxPairs : 1];
  __shared__ double2 s_cs[XF ? kKvWarps : 1][kKvMaxPairs];  // cosine and sine of each pair at the warp's position
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5, sub = lane & (LANES - 1);
  const unsigned int all = LANES == 32 ? 0xffffffffu : 0xffffu << (lane & 16);  // this row's lanes
  // base_rows rows a group of lanes; the first one_more groups take one more
  const int grp = (blockIdx.x * kKvWarps + wib) * (32 / LANES) + lane / LANES;
  const int r0 = grp * base_rows + min(grp, one_more);
  const int r1 = min(a.n_rows, r0 + base_rows + (grp < one_more ? 1 : 0));
  if constexpr (XF) {
    if (a.rotate) {
      for (int j = threadIdx.x; j < k.rope_dims >> 1; j += 32 * kKvWarps)
        s_turn[j] = make_double2(turns.hi[j], turns.lo[j]);
      __syncthreads();
    }
  }
  if (r0 >= r1) return;
  const int nch = k.c >> 3;
  const int rope0 = k.c - k.rope_dims;
  const int n_pairs = XF && a.rotate ? k.rope_dims >> 1 : 0;
  const double inv_c = 1.0 / k.c;
  // The next row is always under way: its load depends on nothing else.
  float next[kU][8];
  auto load_row = [&](int i) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int ch = sub + LANES * u;
      if (ch < nch) {
        load8<F32>(a.x, (long long)i * a.ld_x + ch * 8, next[u]);
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) next[u][t] = 0.f;
      }
    }
  };
  load_row(r0);
  // Request of the first row: the last one that starts at or before it, by a search as wide as the row's lanes.
  int b = r0, start = r0, end = r0 + 1;
  if (a.row_start) {
    int lo = 0, hi = a.B;  // row_start[lo] <= r0 < row_start[hi], if anywhere
    while (hi - lo > 1) {
      const int step = (hi - lo + LANES - 1) / LANES, m = min(lo + sub * step, hi - 1);
      const unsigned int at = (__ballot_sync(all, sub == 0 || a.row_start[m] <= r0) & all) >> (lane & (32 - LANES));
      const int last = 31 - __clz(at);
      hi = min(hi, lo + (last + 1) * step);
      lo = min(lo + last * step, hi - 1);
    }
    b = lo;
    start = a.row_start[b];
    end = a.row_start[b + 1];
  }
  for (int i = r0; i < r1; ++i) {
    float v[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int t = 0; t < 8; ++t) v[u][t] = next[u][t];
    if (i + 1 < r1) load_row(i + 1);
    if (a.row_start) {
      while (i >= end && b + 1 < a.B) {
        ++b;
        start = end;
        end = a.row_start[b + 1];
      }
      if (i < start || i >= end) continue;  // before the first sequence, or behind the last: not appended
    } else {
      b = i;
      start = i;
      end = i + 1;
    }
    const int f = a.first ? a.first[b] : a.first_all;
    const long long e = (long long)f + (i - start);
    if (f < 0) continue;
    if (k.ring && (long long)end - i > k.seq_rows) continue;  // a later row of this call takes its place
    const long long row = e <= 0x7fffffffll ? kv_row(k, b, (int)e) : -1;
    if (row < 0) {
      if (a.check && sub == 0) atomicOr(&g_kv_append_error, 1u);
      continue;
    }
    if constexpr (XF) {
      if (n_pairs > 0) {
        const double pos = (double)((e + 1) * a.rate - 1);
        __syncwarp();  // the last row's table has been read
#pragma unroll 1
        for (int u = 0; 32 * u < n_pairs; ++u) {
          if (lane + 32 * u < n_pairs) {
            const double2 turn = s_turn[lane + 32 * u];
            const double t = pos * turn.x;
            const double rest = fma(pos, turn.y, fma(pos, turn.x, -t));  // what t lacks
            double sn, cs;
            sincospi(2.0 * ((t - rint(t)) + rest), &sn, &cs);
            s_cs[wib][lane + 32 * u] = make_double2(cs, sn);
          }
        }
        __syncwarp();
      }
      double inv = 1.0;
      if (a.gamma) {
        double ss = 0.0;
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int t = 0; t < 8; ++t) ss = fma((double)v[u][t], (double)v[u][t], ss);
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv = rsqrt(fma(ss, inv_c, (double)a.eps));
      }
      // The f32 products below are good to their last bits while nothing overflows or falls to a subnormal: |v| is at most
      // sqrt(c) / inv < 2^45 for an inv of at least 2^-40, |gamma| below 2^60, and a result of at least 2^-80 had factors
      // that were normal.
      const bool narrow = inv >= 0x1p-40 && inv <= 0x1p40;
      const float inv_lo = (float)inv * (1.f - 0x1p-21f), inv_hi = (float)inv * (1.f + 0x1p-21f);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ch = sub + LANES * u;
        if (ch >= nch) continue;
        float g[8];
        if (a.gamma) {
          load8<true>(a.gamma, ch * 8, g);
        } else {
#pragma unroll
          for (int t = 0; t < 8; ++t) g[t] = 1.f;
        }
        if (n_pairs > 0 && 8 * ch >= rope0) {
          const int j0 = (8 * ch - rope0) >> 1;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const double2 r = s_cs[wib][j0 + t];
            const double p = (double)v[u][2 * t] * inv * (double)g[2 * t];
            const double q = (double)v[u][2 * t + 1] * inv * (double)g[2 * t + 1];
            v[u][2 * t] = (float)(p * r.x - q * r.y);
            v[u][2 * t + 1] = (float)(p * r.y + q * r.x);
          }
        } else if (a.gamma) {
          // The value lies between these two f32 products, 8 ulps apart either way; where both round to one bf16, so
          // does it.
          uint32_t w[4], differ = 0;
          float least = 1.f, top = 0.f;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float2 y = mul2(v[u][2 * t], v[u][2 * t + 1], g[2 * t], g[2 * t + 1]);
            const float2 lo = mul2(y.x, y.y, inv_lo, inv_lo), hi = mul2(y.x, y.y, inv_hi, inv_hi);
            w[t] = pack_bf16x2(lo.x, lo.y);
            differ |= w[t] ^ pack_bf16x2(hi.x, hi.y);
            least = fminf(least, fminf(fabsf(lo.x), fabsf(lo.y)));
            top = fmaxf(top, fmaxf(fabsf(g[2 * t]), fabsf(g[2 * t + 1])));
          }
          if (differ || !narrow || least < 0x1p-80f || top > 0x1p60f) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
              w[t] = pack_bf16x2((float)((double)v[u][2 * t] * inv * (double)g[2 * t]),
                                 (float)((double)v[u][2 * t + 1] * inv * (double)g[2 * t + 1]));
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            v[u][2 * t] = bf16_lo(w[t]);
            v[u][2 * t + 1] = bf16_hi(w[t]);
          }
          continue;
        }
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
          const uint32_t w = pack_bf16x2(v[u][t], v[u][t + 1]);
          v[u][t] = bf16_lo(w);
          v[u][t + 1] = bf16_hi(w);
        }
      }
    }
    // the row in the cache's form
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int ch = sub + LANES * u;
      float amax = 0.f;
      if constexpr (FORM != HCA_KV_BF16) {
#pragma unroll
        for (int t = 0; t < 8; ++t) amax = fmaxf(amax, fabsf(v[u][t]));
        amax = fmaxf(amax, __shfl_xor_sync(all, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(all, amax, 2));
        if constexpr (FORM == HCA_KV_FP8) amax = fmaxf(amax, __shfl_xor_sync(all, amax, 4));
      }
      if (ch >= nch) continue;
      const int d = ch * 8;
      if (FORM == HCA_KV_BF16 || d >= rope0) {
        const uint4 w = make_uint4(pack_bf16x2(v[u][0], v[u][1]), pack_bf16x2(v[u][2], v[u][3]),
                                   pack_bf16x2(v[u][4], v[u][5]), pack_bf16x2(v[u][6], v[u][7]));
        bf16* dst = FORM == HCA_KV_BF16 ? reinterpret_cast<bf16*>(k.codes) + row * k.ld_codes + d
                                        : k.rope + row * k.ld_rope + (d - rope0);
        *reinterpret_cast<uint4*>(dst) = w;
      } else if constexpr (FORM == HCA_KV_FP8) {
        const float sc = amax > 0.f ? amax / 448.f : 1.f;
        *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(k.codes) + row * k.ld_codes + d) =
            e4m3x8_encode(v[u], sc);
        if ((ch & 7) == 0) reinterpret_cast<float*>(k.scales)[row * k.ld_scales + ch / 8] = sc;
      } else if constexpr (FORM == HCA_KV_FP4) {
        // scale byte X + 127, X = floor(log2 amax) - 2 in [-127, 127] (an amax of zero or a subnormal gives -127, an
        // infinite one 127), and 2^-X
        const uint32_t ex = __float_as_uint(amax) >> 23, sb = ex == 255u ? 254u : ex > 2u ? ex - 2u : 0u;
        const float down = __uint_as_float(sb < 254u ? (254u - sb) << 23 : 0x00400000u);
        float y[8];
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
          const float2 s = mul2(v[u][t], v[u][t + 1], down, down);
          y[t] = s.x;
          y[t + 1] = s.y;
        }
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(k.codes) + row * k.ld_codes + d / 2) =
            e2m1x8_encode(y);
        if ((ch & 3) == 0) reinterpret_cast<uint8_t*>(k.scales)[row * k.ld_scales + ch / 4] = (uint8_t)sb;
      }
    }
  }
}

// Two E4M3 codes times an f32 scale, in bf16: both are exact in f16 and f32, so the rounding is the product's to f32
// and its to bf16.
__device__ __forceinline__ uint32_t e4m3x2_scaled(uint32_t two, float sc) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(two));
  __half2 v;
  memcpy(&v, &h, 4);
  const float2 f = __half22float2(v);
  return pack_bf16x2(f.x * sc, f.y * sc);
}

// Loads that are made or not (zeros) without a branch, so that a batch of them is under way at once.
__device__ __forceinline__ uint4 load16_if(const void* p, bool ok) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(ok ? 1 : 0));
  return v;
}
__device__ __forceinline__ uint2 load8_if(const void* p, bool ok) {
  uint2 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
      "@p ld.global.v2.b32 {%0, %1}, [%2];\n\t}"
      : "=&r"(v.x), "=&r"(v.y)
      : "l"(p), "r"(ok ? 1 : 0));
  return v;
}
__device__ __forceinline__ uint32_t load4_if(const void* p, bool ok) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.b32 %0, [%1];\n\t}"
               : "=&r"(v)
               : "l"(p), "r"(ok ? 1 : 0));
  return v;
}
__device__ __forceinline__ uint32_t load1_if(const void* p, bool ok) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.u8 %0, [%1];\n\t}"
               : "=&r"(v)
               : "l"(p), "r"(ok ? 1 : 0));
  return v;
}

constexpr int kGatherResident = 5;  // blocks per SM
// Rows in flight per group of LANES lanes, and rows that a block (8 warps) takes at a time.
constexpr int gather_rows(int lanes) { return lanes == 32 ? 2 : 4; }
constexpr int gather_block(int lanes) { return 8 * gather_rows(lanes) * (32 / lanes); }

template <int FORM, int LANES>
__global__ void __launch_bounds__(256, kGatherResident)
    kv_gather_kernel(KvCache k, FastDiv n_out, uint32_t total, const int32_t* __restrict__ idx,
                     const int32_t* __restrict__ first, bf16* __restrict__ out, long long ld_out, long long seq_out) {
  constexpr int kU = LANES == 32 ? kKvChunks : 1;  // chunks per lane
  constexpr int kRows = gather_rows(LANES), kBlock = gather_block(LANES), kStep = 32 / LANES;
  __shared__ long long s_row[2][kBlock], s_dst[2][kBlock];
  const int lane = threadIdx.x & (LANES - 1);
  const int nch = k.c >> 3;
  const int rope0 = k.c - k.rope_dims;
  // Where row o comes from and goes to: one row a thread, 16 dependent chains side by side.
  auto resolve = [&](uint32_t o, int buf) {
    const int b = (int)div_by(o, n_out), j = (int)(o - b * n_out.d);
    int e = j;
    if (idx) {
      e = idx[o];
    } else if (first) {
      const int f = first[b];
      e = f < 0 || f > 0x7fffffff - j ? -1 : f + j;
    }
    s_row[buf][threadIdx.x] = kv_row(k, b, e);
    s_dst[buf][threadIdx.x] = b * seq_out + j * ld_out;
  };
  const uint32_t stride = gridDim.x * kBlock;
  uint32_t base = blockIdx.x * kBlock;
  if (threadIdx.x < kBlock && base + threadIdx.x < total) resolve(base + threadIdx.x, 0);
  __syncthreads();
  for (int buf = 0; base < total; base += stride, buf ^= 1) {
    // (total < 2^31 and the stride is a few thousand rows a time: no overflow)
    if (threadIdx.x < kBlock && base + stride + threadIdx.x < total) resolve(base + stride + threadIdx.x, buf ^ 1);
    {
      const int s0 = (threadIdx.x >> 5) * kRows * kStep + ((threadIdx.x & 31) / LANES);
      long long row[kRows];
      uint4 raw[kU][kRows];
      uint32_t sc[kU][kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) row[r] = base + s0 + r * kStep < total ? s_row[buf][s0 + r * kStep] : -1;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ch = lane + 32 * u, d = ch * 8;
        const bool wide = FORM == HCA_KV_BF16 || d >= rope0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const bool ok = row[r] >= 0 && ch < nch;
          const uint8_t* code = reinterpret_cast<const uint8_t*>(k.codes);
          if constexpr (FORM == HCA_KV_BF16) {
            raw[u][r] = load16_if(code + (row[r] * k.ld_codes + d) * 2, ok);
          } else {
            // lanes of the rotary channels load 16 bytes, the others their codes and scale
            const uint4 w = load16_if(k.rope + row[r] * k.ld_rope + (d - rope0), ok && wide);
            if constexpr (FORM == HCA_KV_FP8) {
              const uint2 t = load8_if(code + row[r] * k.ld_codes + d, ok && !wide);
              raw[u][r] = wide ? w : make_uint4(t.x, t.y, 0u, 0u);
              sc[u][r] = load4_if(reinterpret_cast<const float*>(k.scales) + row[r] * k.ld_scales + ch / 8, ok && !wide);
            } else {
              const uint32_t t = load4_if(code + row[r] * k.ld_codes + d / 2, ok && !wide);
              raw[u][r] = wide ? w : make_uint4(t, 0u, 0u, 0u);
              sc[u][r] = load1_if(reinterpret_cast<const uint8_t*>(k.scales) + row[r] * k.ld_scales + ch / 4, ok && !wide);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ch = lane + 32 * u, d = ch * 8;
        const bool wide = FORM == HCA_KV_BF16 || d >= rope0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (base + s0 + r * kStep >= total || ch >= nch) continue;
          uint4 w = raw[u][r];
          if (!wide && row[r] >= 0) {
            if constexpr (FORM == HCA_KV_FP8) {
              const float s = __uint_as_float(sc[u][r]);
              const uint32_t lo = raw[u][r].x, hi = raw[u][r].y;
              w = make_uint4(e4m3x2_scaled(lo, s), e4m3x2_scaled(lo >> 16, s), e4m3x2_scaled(hi, s),
                             e4m3x2_scaled(hi >> 16, s));
            } else if constexpr (FORM == HCA_KV_FP4) {
              w = e2m1x8_times(raw[u][r].x, e8m0_bf16x2(sc[u][r]));
            }
          }
          *reinterpret_cast<uint4*>(out + s_dst[buf][s0 + r * kStep] + d) = w;
        }
      }
    }
    __syncthreads();
  }
}

// The table for the last base and number of rotary channels used on this thread.
const Turns& turns_of(int rope_dims, float base) {
  static thread_local Turns t;
  static thread_local int have_dims = 0;
  static thread_local float have_base = 0.f;
  if (rope_dims != have_dims || base != have_base) {
    const long double two_pi = 2.0L * acosl(-1.0L);
    for (int j = 0; j < rope_dims / 2; ++j) {
      const long double v = powl((long double)base, -2.0L * j / rope_dims) / two_pi;
      t.hi[j] = (double)v;
      t.lo[j] = (double)(v - (long double)t.hi[j]);
    }
    have_dims = rope_dims;
    have_base = base;
  }
  return t;
}
}  // namespace

template <bool F32, int FORM>
static void append_rows(const KvAppend& a, const KvCache& k, cudaStream_t stream) {
  const bool xf = a.gamma || (a.rotate && k.rope_dims > 0);
  // one row a group of lanes until the machine is full (the resident warps of the launch bounds), then contiguous runs
  const int groups = !xf && k.c <= 128 ? 2 : 1;  // per warp
  const int max_groups = device_sm_count() * kKvWarps * append_blocks(FORM, xf) * groups;
  const int used = std::min(a.n_rows, max_groups), per = a.n_rows / used, more = a.n_rows - per * used;
  const int blocks = (used + kKvWarps * groups - 1) / (kKvWarps * groups);
  const dim3 block(32 * kKvWarps);
  if (xf)
    kv_append_kernel<F32, FORM, true, 32><<<blocks, block, 0, stream>>>(
        a, k, per, more, turns_of(a.rotate ? k.rope_dims : 0, a.rope_base));
  else if (groups == 1) kv_append_kernel<F32, FORM, false, 32><<<blocks, block, 0, stream>>>(a, k, per, more, NoTurns{});
  else kv_append_kernel<F32, FORM, false, 16><<<blocks, block, 0, stream>>>(a, k, per, more, NoTurns{});
}

cudaError_t launch_kv_append(const KvAppend& a, const KvCache& k, cudaStream_t stream) {
  if (a.n_rows <= 0 || a.B <= 0) return cudaSuccess;
  if (k.form == HCA_KV_BF16)
    a.x_f32 ? append_rows<true, HCA_KV_BF16>(a, k, stream) : append_rows<false, HCA_KV_BF16>(a, k, stream);
  else if (k.form == HCA_KV_FP8)
    a.x_f32 ? append_rows<true, HCA_KV_FP8>(a, k, stream) : append_rows<false, HCA_KV_FP8>(a, k, stream);
  else
    a.x_f32 ? append_rows<true, HCA_KV_FP4>(a, k, stream) : append_rows<false, HCA_KV_FP4>(a, k, stream);
  ++g_launch_counter;
  return cudaGetLastError();
}

template <int FORM>
static void gather_rows_of(const KvCache& k, int n_out, long long total, const int32_t* idx, const int32_t* first,
                           bf16* out, long long ld_out, long long seq_out, cudaStream_t stream) {
  const bool narrow = k.c <= 128;  // half a warp a row
  const int block = gather_block(narrow ? 16 : 32);
  const unsigned grid =
      (unsigned)std::min<long long>((total + block - 1) / block, (long long)kGatherResident * device_sm_count());
  const FastDiv n = fast_div((uint32_t)n_out);
  if (narrow)
    kv_gather_kernel<FORM, 16><<<grid, 256, 0, stream>>>(k, n, (uint32_t)total, idx, first, out, ld_out, seq_out);
  else
    kv_gather_kernel<FORM, 32><<<grid, 256, 0, stream>>>(k, n, (uint32_t)total, idx, first, out, ld_out, seq_out);
}

cudaError_t launch_kv_gather(const KvCache& k, int B, int n_out, const int32_t* idx, const int32_t* first, bf16* out,
                             long long ld_out, long long seq_out, cudaStream_t stream) {
  const long long total = (long long)B * n_out;
  if (total <= 0) return cudaSuccess;
  if (k.form == HCA_KV_BF16)
    gather_rows_of<HCA_KV_BF16>(k, n_out, total, idx, first, out, ld_out, seq_out, stream);
  else if (k.form == HCA_KV_FP8)
    gather_rows_of<HCA_KV_FP8>(k, n_out, total, idx, first, out, ld_out, seq_out, stream);
  else
    gather_rows_of<HCA_KV_FP4>(k, n_out, total, idx, first, out, ld_out, seq_out, stream);
  ++g_launch_counter;
  return cudaGetLastError();
}

unsigned int read_and_clear_kv_append_error() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv_append_error, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (v) cudaMemcpyToSymbol(g_kv_append_error, &zero, sizeof(zero));
  return v;
}

}  // namespace hca
