// Shared-KV multi-query attention over a cache in FP4 form (sm_100a).
//
// For query t and head h over the rows U(t) = selected or visible entries, then the window rows:
//   o[t, h, :] = sum_u softmax_u(scale * q[t, h, :] . row_u) row_u
// An entry's row is code * 2^X per 32 channels on its first c - rope_dims channels and bf16 on the rest; both are
// exact in bf16.

#include "common.cuh"
#include "formats.cuh"
#include "internal.h"
#include "tc.cuh"

namespace hca {

__device__ unsigned int g_mqa_fp4_error = 0;

namespace {
// A query's rows: `entries` cache entries (or selected slots), then `window` rows of its request's ring, whose first
// is the row of token tok0.
struct Rows {
  int req, t;
  int entries, window, tok0;
  const int32_t* idx;
};
__device__ __forceinline__ Rows rows_of(const MqaFp4Problem& p, int q) {
  Rows r;
  r.t = p.q_pos[q];
  r.req = p.q_req ? p.q_req[q] : q;
  r.idx = p.idx ? p.idx + (long long)q * p.n_idx : nullptr;
  const bool live = r.t >= 0 && r.req >= 0 && r.req < p.kv.n_req;  // a padding query has no rows
  r.entries = !live || p.N <= 0 ? 0 : (r.idx ? p.n_idx : n_visible(r.t, p.rate, p.N));
  r.tok0 = max(0, r.t - p.n_win + 1);
  r.window = live && p.win ? r.t - r.tok0 + 1 : 0;
  return r;
}
// Cache row of list position u < entries, or -1 for an empty slot.
__device__ __forceinline__ long long entry_row(const MqaFp4Problem& p, const Rows& r, int u) {
  const int e = r.idx ? r.idx[u] : u;
  if (p.check && r.idx) {
    const unsigned int k = entry_check(e, r.t, p.rate, p.N);
    if (k) atomicOr(&g_mqa_fp4_error, k << 1);
  }
  if (e < 0 || e >= p.N) return -1;
  const long long row = kv_row(p.kv, r.req, e);
  if (p.check && row < 0) atomicOr(&g_mqa_fp4_error, kIdxBlock << 1);
  return row;
}
__device__ __forceinline__ const bf16* window_row(const MqaFp4Problem& p, const Rows& r, int w) {
  return p.win + r.req * p.win_seq_stride + (long long)((r.tok0 + w) % p.win_rows) * p.kv.c;
}

// ---- CUDA cores: any c up to 512 ------------------------------------------------------
// One CTA per (query, group of kSH heads, split): rows are widened into shared memory 16 at a time, an online softmax
// runs over them, and the state (m, l, o) goes to the combine kernel.
constexpr int kSThreads = 256, kSRows = 16, kSH = 4;

__global__ void __launch_bounds__(kSThreads) mqa_fp4_simple_kernel(MqaFp4Problem p, int splits, int rows_per_split,
                                                                   float* __restrict__ ws_o,
                                                                   float2* __restrict__ ws_ml) {
  __shared__ float s_q[kSH][512];
  __shared__ __align__(16) bf16 s_r[kSRows][512 + 8];
  __shared__ float s_s[kSH][kSRows];
  __shared__ float s_m[kSH], s_l[kSH], s_a[kSH];
  __shared__ int s_ok[kSRows];
  const int tid = threadIdx.x, c = p.kv.c;
  const int groups = (p.H + kSH - 1) / kSH;
  const int sp = blockIdx.x % splits;
  const int hg = (blockIdx.x / splits) % groups;
  const int q = blockIdx.x / splits / groups;
  const int h0 = hg * kSH, nh = min(kSH, p.H - h0);
  const Rows r = rows_of(p, q);
  const int ub = sp * rows_per_split, ue = min(r.entries + r.window, ub + rows_per_split);
  for (int i = tid; i < kSH * c; i += kSThreads)
    s_q[i / c][i % c] = i / c < nh ? __bfloat162float(p.q[((long long)q * p.H + h0 + i / c) * c + i % c]) : 0.f;
  if (tid < kSH) { s_m[tid] = neg_inf(); s_l[tid] = 0.f; }
  float o[kSH][2] = {};  // channels tid and tid + 256 of each head
  const int n4 = c - p.kv.rope_dims;
  for (int u0 = ub; u0 < ue; u0 += kSRows) {
    __syncthreads();
    for (int i = tid; i < kSRows * (c / 8); i += kSThreads) {
      const int j = i / (c / 8), d = (i % (c / 8)) * 8, u = u0 + j;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      bool ok = false;
      if (u < ue && u < r.entries) {
        const long long row = entry_row(p, r, u);
        ok = row >= 0;
        if (ok && d < n4) {
          uint32_t v[4];
          e2m1x8_to_bf16(*reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(p.kv.codes) +
                                                            row * p.kv.ld_codes + d / 2),
                         (int)reinterpret_cast<const uint8_t*>(p.kv.scales)[row * p.kv.ld_scales + d / 32] - 127, v);
          w = make_uint4(v[0], v[1], v[2], v[3]);
        } else if (ok) {
          w = *reinterpret_cast<const uint4*>(p.kv.rope + row * p.kv.ld_rope + (d - n4));
        }
      } else if (u < ue) {
        ok = true;
        w = *reinterpret_cast<const uint4*>(window_row(p, r, u - r.entries) + d);
      }
      *reinterpret_cast<uint4*>(&s_r[j][d]) = w;
      if (d == 0) s_ok[j] = ok;
    }
    __syncthreads();
    // scores: 4 threads per (head, row)
    {
      const int h = tid / (4 * kSRows), j = (tid >> 2) % kSRows, part = tid & 3;
      float acc = 0.f;
      for (int d = part * 8; d < c; d += 32) {
        float f[8];
        unpack8(*reinterpret_cast<const uint4*>(&s_r[j][d]), f);
#pragma unroll
        for (int t = 0; t < 8; ++t) acc = fmaf(s_q[h][d + t], f[t], acc);
      }
      acc += __shfl_xor_sync(0xffffffffu, acc, 1);
      acc += __shfl_xor_sync(0xffffffffu, acc, 2);
      if (part == 0) s_s[h][j] = s_ok[j] ? acc * (p.scale * kLog2e) : neg_inf();
    }
    __syncthreads();
    if (tid < kSH) {
      float mn = s_m[tid];
      for (int j = 0; j < kSRows; ++j) mn = fmaxf(mn, s_s[tid][j]);
      const float alpha = mn == neg_inf() ? 1.f : fast_exp2(s_m[tid] - mn);
      float l = s_l[tid] * alpha;
      for (int j = 0; j < kSRows; ++j) {
        const float e = mn == neg_inf() ? 0.f : fast_exp2(s_s[tid][j] - mn);
        s_s[tid][j] = e;
        l += e;
      }
      s_m[tid] = mn;
      s_l[tid] = l;
      s_a[tid] = alpha;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kSH; ++h) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = tid + k * kSThreads;
        if (d >= c) continue;
        float acc = o[h][k] * s_a[h];
        for (int j = 0; j < kSRows; ++j) acc = fmaf(s_s[h][j], __bfloat162float(s_r[j][d]), acc);
        o[h][k] = acc;
      }
    }
  }
  __syncthreads();
  const long long st = (long long)q * splits + sp;
#pragma unroll
  for (int h = 0; h < kSH; ++h) {
    if (h >= nh) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = tid + k * kSThreads;
      if (d < c) ws_o[(st * p.H + h0 + h) * c + d] = o[h][k];
    }
  }
  if (tid < nh) ws_ml[st * p.H + h0 + tid] = make_float2(s_m[tid], s_l[tid]);
}
}  // namespace

MqaPlan plan_mqa_fp4(const MqaFp4Problem& p, int num_sms) {
  MqaPlan pl;
  pl.max_rows = max(1, (p.idx ? p.n_idx : p.N) + (p.win ? p.n_win : 0));
  const int groups = (p.H + kSH - 1) / kSH;
  int splits = (int)max(1ll, (8ll * num_sms) / max(1ll, (long long)p.Tq * groups));
  splits = min(min(splits, 64), (pl.max_rows + kSRows - 1) / kSRows);
  pl.rows_per_split = ((pl.max_rows + splits - 1) / splits + kSRows - 1) / kSRows * kSRows;
  pl.splits = (pl.max_rows + pl.rows_per_split - 1) / pl.rows_per_split;
  pl.ws_bytes = (size_t)p.Tq * pl.splits * p.H * ((size_t)p.kv.c * sizeof(float) + sizeof(float2));
  return pl;
}

cudaError_t launch_mqa_fp4(const MqaFp4Problem& p, const MqaPlan& pl, void* ws, cudaStream_t stream) {
  if (p.Tq == 0) return cudaSuccess;
  float* ws_o = reinterpret_cast<float*>(ws);
  float2* ws_ml = reinterpret_cast<float2*>(ws_o + (size_t)p.Tq * pl.splits * p.H * p.kv.c);
  const int groups = (p.H + kSH - 1) / kSH;
  mqa_fp4_simple_kernel<<<(unsigned)(p.Tq * groups * pl.splits), kSThreads, 0, stream>>>(p, pl.splits,
                                                                                        pl.rows_per_split, ws_o, ws_ml);
  ++g_launch_counter;
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_mqa_combine(ws_o, ws_ml, p.Tq, pl.splits, p.H, p.kv.c, p.out, p.sink, p.q_pos, p.rope_dims, p.rope_base,
                            stream, true);
}

unsigned int read_and_clear_mqa_fp4_error() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_mqa_fp4_error, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (v) cudaMemcpyToSymbol(g_mqa_fp4_error, &zero, sizeof(zero));
  return v;
}

}  // namespace hca
