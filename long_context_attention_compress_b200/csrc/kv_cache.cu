// Rows into and out of a KV cache held in bf16, FP8 or FP4, flat, paged or a ring (sm_100a).
//
// kv_append_kernel.  y = x, or bf16(R_pos(x / sqrt(mean(x^2) + eps) * gamma)) with pos = (entry + 1)*rate - 1 and R
// the rotation of the last rope_dims channels; then y in the cache's form:
//   bf16; FP8: scale = f32(amax / 448) per 64 channels, the E4M3 value nearest to y / scale; FP4: 2^X per 32
//   channels, X = floor(log2 amax) - 2, the E2M1 value nearest to y * 2^-X; the last rope_dims channels bf16.
// One warp owns a row: lane l holds the 8-channel chunks l and l + 32, so a group's maximum is two (FP4) or three
// (FP8) shuffles away and nothing passes through memory between the input and the stored row.  Bound by HBM for many
// rows (c*4 B in, 366 B out for FP4 at c = 512), by latency for few.
// Roundings.  With normalisation or rotation y is rounded to bf16 first (what the bf16 cache holds), as from the
// float64 value: a quantised code must not depend on which side of a midpoint an f32 normalisation falls.  Sum of
// squares and rotation are f64; the other channels are formed in f32 and redone in f64 only within 16 f32 ulps of a
// bf16 midpoint (f32 is within 3).  The codes are those of the stored-form definitions bit for bit: FP4 scaling is
// exact and the conversion rounds to nearest even; an f32 quotient within 4 ulps of an E4M3 midpoint, or in E4M3's
// subnormal range, is decided on the f64 quotient.
//
// kv_gather_kernel.  The bf16 values of rows; one warp a row, four rows in flight per warp (each row is a chain of
// dependent loads: index, block table, row).

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

// Two E4M3 codes of y / sc (see the head of this file).
__device__ __forceinline__ bool e4m3_doubtful(float q) {
  const int low = (int)(__float_as_uint(q) & 0xfffffu) - 0x80000;
  return !(fabsf(q) >= 0.015625f) || (low >= -4 && low <= 4);
}
__device__ __forceinline__ uint32_t e4m3x2_encode(float y0, float y1, float sc) {
  const float q0 = y0 / sc, q1 = y1 / sc;
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(q1), "f"(q0));
  uint32_t w = h;
  if (e4m3_doubtful(q0)) w = (w & 0xff00u) | e4m3_encode((double)y0 / (double)sc);
  if (e4m3_doubtful(q1)) w = (w & 0x00ffu) | (e4m3_encode((double)y1 / (double)sc) << 8);
  return w;
}

template <bool F32, int FORM>
__global__ void __launch_bounds__(32 * kKvWarps) kv_append_kernel(KvAppend a, KvCache k, int rows_per_warp) {
  __shared__ double2 s_cs[kKvWarps][kKvMaxPairs];  // cosine and sine of each pair at the warp's current position
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  const int r0 = (blockIdx.x * kKvWarps + wib) * rows_per_warp;
  const int r1 = min(a.n_rows, r0 + rows_per_warp);
  if (r0 >= r1) return;
  const int nch = k.c >> 3;
  const int rope0 = k.c - k.rope_dims;
  const int n_pairs = a.rotate ? k.rope_dims >> 1 : 0;
  double theta[kKvMaxPairs / 32];
#pragma unroll
  for (int u = 0; u < kKvMaxPairs / 32; ++u)
    theta[u] = lane + 32 * u < n_pairs ? pow((double)a.rope_base, -2.0 * (lane + 32 * u) / k.rope_dims) : 0.0;
  // request of the first row: the last one that starts at or before it
  int b = r0, start = r0, end = r0 + 1;
  if (a.row_start) {
    int lo = 0, hi = a.B;  // row_start[lo] <= r0 < row_start[hi], if anywhere
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.row_start[mid] <= r0) lo = mid; else hi = mid;
    }
    b = lo;
    start = a.row_start[b];
    end = a.row_start[b + 1];
  }
  for (int i = r0; i < r1; ++i) {
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
    const long long row = kv_row(k, b, e);
    if (row < 0) {
      if (a.check && lane == 0) atomicOr(&g_kv_append_error, 1u);
      continue;
    }
    float v[kKvChunks][8];
#pragma unroll
    for (int u = 0; u < kKvChunks; ++u) {
      const int ch = lane + 32 * u;
      if (ch < nch) {
        load8<F32>(a.x, (long long)i * a.ld_x + ch * 8, v[u]);
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) v[u][t] = 0.f;
      }
    }
    if (n_pairs > 0) {
      const double pos = (double)((e + 1) * a.rate - 1);
      __syncwarp();  // the last row's table has been read
#pragma unroll
      for (int u = 0; u < kKvMaxPairs / 32; ++u) {
        if (lane + 32 * u < n_pairs) {
          double sn, cs;
          sincos(pos * theta[u], &sn, &cs);
          s_cs[wib][lane + 32 * u] = make_double2(cs, sn);
        }
      }
      __syncwarp();
    }
    if (a.gamma || n_pairs > 0) {
      double inv = 1.0;
      if (a.gamma) {
        double ss = 0.0;
#pragma unroll
        for (int u = 0; u < kKvChunks; ++u)
#pragma unroll
          for (int t = 0; t < 8; ++t) ss = fma((double)v[u][t], (double)v[u][t], ss);
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv = rsqrt(ss / k.c + (double)a.eps);
      }
      const float inv32 = (float)inv;
#pragma unroll
      for (int u = 0; u < kKvChunks; ++u) {
        const int ch = lane + 32 * u;
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
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            float y = v[u][t] * inv32 * g[t];
            const int low = (int)(__float_as_uint(y) & 0xffffu) - 0x8000;  // 0: a bf16 midpoint
            if (low > -16 && low < 16) y = (float)((double)v[u][t] * inv * (double)g[t]);
            v[u][t] = y;
          }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) v[u][t] = __bfloat162float(__float2bfloat16_rn(v[u][t]));
      }
    }
    // the row in the cache's form
#pragma unroll
    for (int u = 0; u < kKvChunks; ++u) {
      const int ch = lane + 32 * u;
      float amax = 0.f;
      if constexpr (FORM != HCA_KV_BF16) {
#pragma unroll
        for (int t = 0; t < 8; ++t) amax = fmaxf(amax, fabsf(v[u][t]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if constexpr (FORM == HCA_KV_FP8) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
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
        uint2 w;
        w.x = e4m3x2_encode(v[u][0], v[u][1], sc) | (e4m3x2_encode(v[u][2], v[u][3], sc) << 16);
        w.y = e4m3x2_encode(v[u][4], v[u][5], sc) | (e4m3x2_encode(v[u][6], v[u][7], sc) << 16);
        *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(k.codes) + row * k.ld_codes + d) = w;
        if ((ch & 7) == 0) reinterpret_cast<float*>(k.scales)[row * k.ld_scales + ch / 8] = sc;
      } else if constexpr (FORM == HCA_KV_FP4) {
        const int X = mx_exponent(amax);
        const float down = __uint_as_float(X < 127 ? (uint32_t)(127 - X) << 23 : 0x00400000u);  // 2^-X
        float y[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) y[t] = v[u][t] * down;
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(k.codes) + row * k.ld_codes + d / 2) =
            e2m1x8_encode(y);
        if ((ch & 3) == 0) reinterpret_cast<uint8_t*>(k.scales)[row * k.ld_scales + ch / 4] = (uint8_t)(X + 127);
      }
    }
  }
}

// E4M3 byte times an f32 scale (one rounding, in the product): the magnitude's bits, seen as an f32 2^120 too
// small, are exact for subnormal codes too.
__device__ __forceinline__ float e4m3_scaled(uint32_t b, float sc) {
  const float mag = __uint_as_float((b & 0x7fu) << 20) * 1.329227995784916e36f;  // 2^120
  return ((b & 0x80u) ? -mag : mag) * sc;
}

constexpr int kGatherRows = 4;  // rows in flight per warp

template <int FORM>
__global__ void __launch_bounds__(256) kv_gather_kernel(KvCache k, int n_out, long long total,
                                                        const int32_t* __restrict__ idx,
                                                        const int32_t* __restrict__ first, bf16* __restrict__ out,
                                                        long long ld_out, long long seq_out) {
  const int lane = threadIdx.x & 31;
  const long long w0 = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int nch = k.c >> 3;
  const int rope0 = k.c - k.rope_dims;
  long long row[kGatherRows], dst[kGatherRows];
#pragma unroll
  for (int r = 0; r < kGatherRows; ++r) {
    const long long o = w0 * kGatherRows + r;
    row[r] = -1;
    dst[r] = -1;
    if (o < total) {
      const int b = (int)(o / n_out), j = (int)(o % n_out);
      long long e = j;
      if (idx) {
        e = idx[o];
      } else if (first) {
        const int f = first[b];
        e = f < 0 ? -1 : (long long)f + j;
      }
      row[r] = kv_row(k, b, e);
      dst[r] = b * seq_out + j * ld_out;
    }
  }
#pragma unroll
  for (int u = 0; u < kKvChunks; ++u) {
    const int ch = lane + 32 * u, d = ch * 8;
    if (ch >= nch) continue;
    const bool wide = FORM == HCA_KV_BF16 || d >= rope0;
    uint4 raw[kGatherRows];
    uint32_t sc[kGatherRows];
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
      raw[r] = make_uint4(0u, 0u, 0u, 0u);
      sc[r] = 0u;
      if (row[r] < 0) continue;
      if (wide) {
        raw[r] = *reinterpret_cast<const uint4*>(
            FORM == HCA_KV_BF16 ? reinterpret_cast<const bf16*>(k.codes) + row[r] * k.ld_codes + d
                                : k.rope + row[r] * k.ld_rope + (d - rope0));
      } else if constexpr (FORM == HCA_KV_FP8) {
        const uint2 t = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(k.codes) +
                                                        row[r] * k.ld_codes + d);
        raw[r].x = t.x;
        raw[r].y = t.y;
        sc[r] = __float_as_uint(reinterpret_cast<const float*>(k.scales)[row[r] * k.ld_scales + ch / 8]);
      } else if constexpr (FORM == HCA_KV_FP4) {
        raw[r].x = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(k.codes) +
                                                      row[r] * k.ld_codes + d / 2);
        sc[r] = reinterpret_cast<const uint8_t*>(k.scales)[row[r] * k.ld_scales + ch / 4];
      }
    }
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
      if (dst[r] < 0) continue;
      uint4 w = raw[r];
      if (!wide && row[r] >= 0) {
        if constexpr (FORM == HCA_KV_FP8) {
          const float s = __uint_as_float(sc[r]);
          const uint32_t lo = raw[r].x, hi = raw[r].y;
          w.x = pack_bf16x2(e4m3_scaled(lo, s), e4m3_scaled(lo >> 8, s));
          w.y = pack_bf16x2(e4m3_scaled(lo >> 16, s), e4m3_scaled(lo >> 24, s));
          w.z = pack_bf16x2(e4m3_scaled(hi, s), e4m3_scaled(hi >> 8, s));
          w.w = pack_bf16x2(e4m3_scaled(hi >> 16, s), e4m3_scaled(hi >> 24, s));
        } else if constexpr (FORM == HCA_KV_FP4) {
          uint32_t o[4];
          e2m1x8_to_bf16(raw[r].x, (int)sc[r] - 127, o);
          w = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      *reinterpret_cast<uint4*>(out + dst[r] + d) = w;
    }
  }
}
}  // namespace

template <bool F32>
static void append_form(const KvAppend& a, const KvCache& k, unsigned grid, int per, cudaStream_t stream) {
  if (k.form == HCA_KV_BF16)
    kv_append_kernel<F32, HCA_KV_BF16><<<grid, 32 * kKvWarps, 0, stream>>>(a, k, per);
  else if (k.form == HCA_KV_FP8)
    kv_append_kernel<F32, HCA_KV_FP8><<<grid, 32 * kKvWarps, 0, stream>>>(a, k, per);
  else
    kv_append_kernel<F32, HCA_KV_FP4><<<grid, 32 * kKvWarps, 0, stream>>>(a, k, per);
}

cudaError_t launch_kv_append(const KvAppend& a, const KvCache& k, cudaStream_t stream) {
  if (a.n_rows <= 0 || a.B <= 0) return cudaSuccess;
  // one row a warp until the machine is full (32 warps per SM), then contiguous runs
  const int max_warps = device_sm_count() * 32;
  const int per = (a.n_rows + max_warps - 1) / max_warps;
  const int warps = (a.n_rows + per - 1) / per;
  const unsigned grid = (unsigned)((warps + kKvWarps - 1) / kKvWarps);
  if (a.x_f32) append_form<true>(a, k, grid, per, stream);
  else append_form<false>(a, k, grid, per, stream);
  ++g_launch_counter;
  return cudaGetLastError();
}

cudaError_t launch_kv_gather(const KvCache& k, int B, int n_out, const int32_t* idx, const int32_t* first, bf16* out,
                             long long ld_out, long long seq_out, cudaStream_t stream) {
  const long long total = (long long)B * n_out;
  if (total <= 0) return cudaSuccess;
  const unsigned grid = (unsigned)((total + 8 * kGatherRows - 1) / (8 * kGatherRows));
  if (k.form == HCA_KV_BF16)
    kv_gather_kernel<HCA_KV_BF16><<<grid, 256, 0, stream>>>(k, n_out, total, idx, first, out, ld_out, seq_out);
  else if (k.form == HCA_KV_FP8)
    kv_gather_kernel<HCA_KV_FP8><<<grid, 256, 0, stream>>>(k, n_out, total, idx, first, out, ld_out, seq_out);
  else
    kv_gather_kernel<HCA_KV_FP4><<<grid, 256, 0, stream>>>(k, n_out, total, idx, first, out, ld_out, seq_out);
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
