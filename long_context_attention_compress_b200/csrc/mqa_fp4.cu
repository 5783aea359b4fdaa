// Shared-KV multi-query attention over a cache in FP4 form (sm_100a).
//
// For query t and head h over the rows U(t) = selected or visible entries, then the window rows:
//   o[t, h, :] = sum_u softmax_u(scale * q[t, h, :] . row_u) row_u
// An entry's row is code * 2^X per 32 channels on its first c - rope_dims channels and bf16 on the rest; both are
// exact in bf16.
//
// Work: a row is 366 bytes at c = 512 (56 ps of HBM time) and 4*H*c flops a query (78 ps of tensor time at 64 heads),
// once widened.  Widening is what the two do not show: 14 half-rate byte permutes and 4 multiplies per 8 codes, 1.8 k
// cycles of an SM's four ALUs per 128 rows, against 0.9 k for the flops at full rate.
// Roundings: products are exact in f32 and summed in f32 by the tensor cores; logits, softmax, states and sums are f32.
// P enters the second product as P_hi + P_lo, P_hi truncated to bf16 and P_lo the rest rounded to bf16 (within 2^-15 of
// P), and the row sums are those of what is multiplied: the output's rounding to bf16 (1.7e-3) is the only one that
// shows.  P_hi alone left 2.2e-3.

#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "formats.cuh"
#include "internal.h"
#include "tc.cuh"

namespace hca {

__device__ unsigned int g_mqa_fp4_error = 0;

namespace {
// Entries of N that a query at position t >= 0 sees (t + 1 as an unsigned number: positions go up to 2^31 - 1).
__device__ __forceinline__ int entries_seen(int t, int rate, int N) {
  return (int)min(((uint32_t)t + 1u) / (uint32_t)rate, (uint32_t)N);
}
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
  r.entries = !live || p.N <= 0 ? 0 : (r.idx ? p.n_idx : entries_seen(r.t, p.rate, p.N));
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

// ---- CUDA cores: c other than 512 ------------------------------------------------------
// One CTA per (query, group of kSH heads, split): rows are widened into shared memory 16 at a time, an online softmax
// runs over them, and the state (m, l, o) goes to the combine kernel.  Bound by f32 FMAs and shared memory: it took
// 1.2 ms for the 8 x 8,192 entries of c = 512 that take 37.3 us below; the small widths it serves are short.
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
      // (the maximum takes no account of a NaN, but its row's weight is one; a maximum of -inf, no row yet or none with a
      // finite score, leaves weights of 0 and NaN)
      float mn = s_m[tid];
      for (int j = 0; j < kSRows; ++j) mn = fmaxf(mn, s_s[tid][j]);
      const float ref = mn == neg_inf() ? 0.f : mn;
      const float alpha = fast_exp2(s_m[tid] - ref);  // (0 before the first row, whose sums are 0)
      float l = s_l[tid] * alpha;
      for (int j = 0; j < kSRows; ++j) {
        const float e = fast_exp2(s_s[tid][j] - ref);
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

// ---- tcgen05: c = 512 -------------------------------------------------------------------
// Rows are the MMA's M dimension and heads its N dimension (64 heads a CTA; fewer are padded with zero queries):
// a 128-row tile, widened to bf16 in shared memory (128B-swizzled, eight 64-channel chunks), is the K-major A operand
// of S^T = R . Q^T and, read MN-major, the A operand of O^T += V^T . P^T.  It is tracked as four 128-channel blocks:
// PV releases them one by one, the converters refill them with the next tile, and QK^T of that tile follows block by
// block.
//   warp 0        MMA issuer (and TMEM owner); warps 1-3 only complete its warpgroup
//   warps 4-11    softmax: two per TMEM lane quarter (32 rows), 32 heads each; P = 2^(s - m) as two bf16 terms,
//                 the row sums in f32 from those, formed after P has been handed over; accumulators rescaled only
//                 when some score exceeds its head's running reference by 20 (in log2)
//   warps 12-27   converters: eight rows a warp, thread = (row, one of a block's four 32-channel groups), so that a
//                 warp's load touches eight rows' lines, not 32; the next tile's codes are loaded and widened into
//                 registers while QK^T and the softmax run, so that only stores lie between PV releasing a block
//                 and the next QK^T over it; rotary channels go the same way without widening (their lines are
//                 brought to L2 a tile ahead), window rows are copied with 16-byte cp.async
// Where few heads would leave columns empty, they are given to neighbouring queries (see Group below).
//
// Measured at 64 heads: 8 requests x 8,192 entries 37.3 us, 32 x 1,024 selected 31.8 us; 16 heads, 2 x 192 queries over
// 2,900 entries 113 us.  With P as one bf16 term they took 33.6, 29.3 and 101 us, and the outputs were off by a third
// more than their own rounding.  Steady state, every SM at work: 8.8 k cycles a tile (7.3 k with one term): the softmax,
// then PV (2.3 k: 288 KiB of operands at the shared-memory rate), the blocks' refill (128 KiB of stores) beside PV's end
// and QK^T (192 KiB).  Around it 11.5 k cycles before the first P (set-up, the chain q_pos - block table - codes, one
// tile's widening) and 5 k for 128 KiB of partial states (26 B a cycle and SM, the rate of L2 writes), then the combine.
// Tried and dropped: QK^T from rows in TMEM with V's stores behind PV (the converters' work comes in series, or their
// loads touch 32 rows each: 45 and 37.5 us where this took 33.6); one proxy fence for several blocks, the widening held
// back until P is signalled, the E2M1 conversion instruction for half of the codes, all four blocks widened ahead (no
// gain or slower).
constexpr int kSoft = 8, kConv = 16;
constexpr int kThreads = 32 * (4 + kSoft + kConv);   // whole warpgroups, for the register split
constexpr int kRowsT = 128;                          // rows per tile
constexpr int kC = 512, kHT = 64;                    // channels; heads per CTA
constexpr int kBlocks = 4;                           // 128-channel blocks of a tile
constexpr uint32_t kQChunk = kHT * 128;              // 8 KiB: 64 channels of the queries
constexpr uint32_t kKvChunk = kRowsT * 128;          // 16 KiB: 64 channels of the tile
constexpr uint32_t kQBytes = 8 * kQChunk, kKvBytes = 8 * kKvChunk, kPBytes = kRowsT * kHT * 2;
constexpr uint32_t kOffQ = 0, kOffKv = kQBytes, kOffP = kOffKv + kKvBytes, kOffBars = kOffP + 2 * kPBytes;
// TMEM: S^T, then O^T block by block.  Blocks 0-2 keep the products with P_hi and P_lo apart (128 columns: one N = 128
// MMA reads the rows once for both); the last block, whose 64 columns are what is left, takes them one after the other.
constexpr uint32_t kColS = 0, kColO = 64, kColBlock = 2 * kHT, kTmemCols = 512;
constexpr float kRescaleLog2 = 20.f;
constexpr float kNoMax = -3.4028234663852886e38f;     // running maximum of a head without a score yet: f32's least
// A reference is a scaled score rounded down.  Scaled scores minus their reference are one FMA, whose product is exact:
// what the reference was rounded by, less than 8 below this magnitude, stays in every weight of the head and cancels.
// Above it, it could pass the exponential's range: there every product is rounded as the reference was (see write_p).
constexpr float kLarge = 0x1p27f;
constexpr int kHpt = kHT * 4 / kSoft;                // heads per softmax thread (32)
constexpr int kOutLd = kC + 8;                       // staged output row (bf16), padded against bank conflicts

struct __align__(16) Bars {
  float red[4][kHT];
  float nref[kHT];      // running maxima, negated
  float alpha[kHT];
  uint64_t qfull, vfull[kBlocks], vempty[kBlocks], sfull, pfull, odone, drain;
  uint32_t rowok[4][kConv];  // [tile % 4][converter warp]: bit 4 j is set where row j of the warp's eight takes part
  uint32_t tmem_base;
  alignas(8) int abort;
  int large;             // some head's reference is kLarge or more in magnitude (read together with abort)
};
constexpr size_t kSmemBytes = 1024 + kOffBars + sizeof(Bars);
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kHT * kOutLd * 2 <= kKvBytes, "staged output fits in the tile buffer");

// One reduce-scatter step over lane bit O: of the NV values held, keep the half selected by the bit and add the
// partner's copy of that half.
template <int O, int NV>
__device__ __forceinline__ void rs_sum_step(float (&a)[16], int lane) {
  const bool hi = (lane & O) != 0;
#pragma unroll
  for (int j = 0; j < NV / 2; ++j) {
    const float send = hi ? a[j] : a[j + NV / 2];
    const float keep = hi ? a[j + NV / 2] : a[j];
    a[j] = keep + __shfl_xor_sync(0xffffffffu, send, O);
  }
}
// Afterwards lane l holds the warp-wide sum of value l % 16.
__device__ __forceinline__ float warp_sum16(float (&a)[16], int lane) {
  rs_sum_step<8, 16>(a, lane);
  rs_sum_step<4, 8>(a, lane);
  rs_sum_step<2, 4>(a, lane);
  rs_sum_step<1, 2>(a, lane);
  return a[0] + __shfl_xor_sync(0xffffffffu, a[0], 16);
}
// Whether one of eight bf16 values is an infinity or a NaN.
__device__ __forceinline__ bool any_not_finite(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool r = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) r |= (w[k] & 0x7f80u) == 0x7f80u || (w[k] & 0x7f800000u) == 0x7f800000u;
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// What a CTA attends to.  Without packing: one query and up to 64 of its heads.  Packed (dense entries, at most 32
// heads, several queries a request): the 64 columns of the MMA are the heads of G consecutive queries (see mqa_fp4_pack),
// so that the queries of a chunk share the rows that are widened for them.  The group is cut into runs
// of neighbouring queries of one request with positions at most kRunStep apart; a run's rows are the union of its
// queries', and each column masks the rows that its query does not see.
constexpr int kRunStep = 4;
struct Run {
  int j0, j1;         // queries of the group
  int req;
  int entries;        // cache entries (or selected slots)
  int tok0, window;   // window tokens tok0 .. tok0 + window - 1
  int na, n;          // tiles of entries, and all
  int least;          // entries that every query of the run sees
};
template <bool PACK>
struct Group {
  int n;              // queries
  int t, vis, req;    // this lane's query: position (-1: a padding query), entries, request
  unsigned int starts;
  const int32_t* idx;
  __device__ __forceinline__ Group(const MqaFp4Problem& p, int q0, int g, int lane) {
    n = PACK ? min(g, p.Tq - q0) : 1;
    const int j = PACK ? min(lane, n - 1) : 0;
    t = p.q_pos[q0 + j];
    req = p.q_req ? p.q_req[q0 + j] : q0 + j;
    idx = p.idx ? p.idx + (long long)q0 * p.n_idx : nullptr;
    if (t < 0 || req < 0 || req >= p.kv.n_req) t = -1;
    vis = t < 0 || p.N <= 0 ? 0 : (idx ? p.n_idx : entries_seen(t, p.rate, p.N));
    starts = 1u;
    if (PACK) {
      const int t1 = __shfl_up_sync(0xffffffffu, t, 1), r1 = __shfl_up_sync(0xffffffffu, req, 1);
      starts = __ballot_sync(0xffffffffu, lane == 0 || r1 != req || (t1 < 0) != (t < 0) || t - t1 > kRunStep ||
                                              t1 - t > kRunStep);
    }
  }
  // (all lanes of a warp)
  __device__ __forceinline__ Run run(const MqaFp4Problem& p, int j0, int lane) const {
    Run r;
    r.j0 = j0;
    r.j1 = 1;
    int tmin = t, tmax = t;
    r.entries = r.least = vis;
    r.req = req;
    if (PACK) {
      const unsigned int later = j0 < 31 ? starts >> (j0 + 1) : 0u;
      r.j1 = min(n, later ? j0 + __ffs(later) : 32);
      const bool in = lane >= r.j0 && lane < r.j1;
      r.entries = __reduce_max_sync(0xffffffffu, in ? vis : 0);
      r.least = __reduce_min_sync(0xffffffffu, in ? vis : 0x7fffffff);
      tmin = __reduce_min_sync(0xffffffffu, in ? t : 0x7fffffff);
      tmax = __reduce_max_sync(0xffffffffu, in ? t : -1);
      r.req = __shfl_sync(0xffffffffu, req, j0);
    }
    r.tok0 = max(0, tmin - p.n_win + 1);
    r.window = tmax >= 0 && p.win ? tmax - r.tok0 + 1 : 0;
    r.na = (r.entries + kRowsT - 1) / kRowsT;
    r.n = r.na + (r.window + kRowsT - 1) / kRowsT;
    return r;
  }
};

template <bool PACK>
__global__ void __launch_bounds__(kThreads, 1) mqa_fp4_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                                 MqaFp4Problem p, int G, int splits,
                                                                 float* __restrict__ ws_o,
                                                                 float2* __restrict__ ws_ml) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = tc::smem_align1024(smem_raw);
  Bars* bars = reinterpret_cast<Bars*>(base + kOffBars);
  volatile int* abort = &bars->abort;
  volatile unsigned long long* abort_or_large = reinterpret_cast<volatile unsigned long long*>(&bars->abort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sp = blockIdx.x % splits;
  const int heads = PACK ? 1 : (p.H + kHT - 1) / kHT;  // groups of 64 heads
  const int h0 = PACK ? 0 : ((blockIdx.x / splits) % heads) * kHT;
  const int q0 = blockIdx.x / splits / heads * (PACK ? G : 1);
  const Group<PACK> grp(p, q0, G, lane);  // (its loads overlap the set-up below)

  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->qfull, 1);
    for (int b = 0; b < kBlocks; ++b) {
      tc::mbar_init(&bars->vfull[b], kConv);
      tc::mbar_init(&bars->vempty[b], 1);
    }
    tc::mbar_init(&bars->sfull, 1);
    tc::mbar_init(&bars->pfull, kSoft);
    tc::mbar_init(&bars->odone, 1);
    tc::mbar_init(&bars->drain, 1);
    bars->abort = 0;
    bars->large = 0;
    tc::fence_mbar_init();
  }
  for (int h = threadIdx.x; h < kHT; h += kThreads) bars->nref[h] = -kNoMax;
  if (warp == 0) tc::tmem_alloc(&bars->tmem_base, kTmemCols);
  // The group's tiles, run by run, entries before the window; this CTA takes those from ga to gb.
  int total = 0;
  for (int j = 0; j < grp.n;) {
    const Run r = grp.run(p, j, lane);
    total += r.n;
    j = r.j1;
  }
  const int each = total / splits, extra = total - each * splits;  // the first `extra` CTAs take one more
  const int ga = sp * each + min(sp, extra), nt = each + (sp < extra ? 1 : 0), gb = ga + nt;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  tc::griddep_launch_dependents();

  // ---- epilogue pieces, shared by the softmax and converter warps ----
  // Row of the partial states (or, unsplit, of the output) of column lane and of column 32 + lane; -1: not an output.
  auto column_row = [&](int c) -> int {
    if (PACK) {
      const int j = c / p.H;
      return j < grp.n ? ((q0 + j) * splits + sp) * p.H + (c - j * p.H) : -1;
    }
    return h0 + c < p.H ? (q0 * splits + sp) * p.H + h0 + c : -1;
  };
  const int quarter = warp & 3;  // TMEM lanes of this warp
  const uint32_t lanebase = (uint32_t)(quarter * 32) << 16;
  bf16* stage = reinterpret_cast<bf16*>(base + kOffKv);  // the last PV has read the tile
  // Channels [128 b + 32 quarter, +32) of columns [16 x, 16 x + 16): partial states to memory, or the finished output,
  // turned by (rc, rs), to its staging.
  auto store_part = [&](int b, int x, float rc, float rs) {
    uint32_t v[16];
    if (nt > 0) {
      tc::tmem_ld16(tmem + lanebase + kColO + b * kColBlock + 16 * x, v);
      if (b < kBlocks - 1) {
        uint32_t lo[16];
        tc::tmem_ld16(tmem + lanebase + kColO + b * kColBlock + kHT + 16 * x, lo);
        tc::tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 16; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) + __uint_as_float(lo[h]));
      } else {
        tc::tmem_ld_wait();
      }
    } else {
#pragma unroll
      for (int h = 0; h < 16; ++h) v[h] = 0u;
    }
    const int d = b * 128 + quarter * 32 + lane;
    if (PACK || splits > 1) {
      const int mine = column_row(32 * (x >> 1) + lane);
#pragma unroll
      for (int h = 0; h < 16; ++h) {
        const int to = __shfl_sync(0xffffffffu, mine, 16 * (x & 1) + h);
        if (to >= 0) ws_o[(long long)to * kC + d] = __uint_as_float(v[h]);
      }
      return;
    }
    const bool rot = p.rope_dims > 0 && b * 128 + quarter * 32 + 31 >= kC - p.rope_dims;  // (of whole warps)
#pragma unroll
    for (int h = 0; h < 16; ++h) {
      const float inv = bars->alpha[16 * x + h];
      float o = __uint_as_float(v[h]) * inv;  // (no rows: 0 * 0; rows of weight 0 that are not finite show)
      if (rot) o = fmaf(o, rc, __shfl_xor_sync(0xffffffffu, o, 1) * rs);
      stage[(16 * x + h) * kOutLd + d] = __float2bfloat16_rn(o);
    }
  };
  // After every softmax and converter warp has staged its parts: the output's rows, 16 bytes a thread.
  auto copy_out = [&]() {
    if (PACK || splits > 1) return;
    tc::named_bar(3, 32 * (kSoft + kConv));
    bf16* out = p.out + ((long long)q0 * p.H + h0) * kC;
    const int nh = min(kHT, p.H - h0);
    for (int u = threadIdx.x - 128; u < nh * (kC / 8); u += 32 * (kSoft + kConv)) {
      const int h = u / (kC / 8), x = u % (kC / 8);
      *reinterpret_cast<uint4*>(out + h * kC + x * 8) = *reinterpret_cast<const uint4*>(stage + h * kOutLd + x * 8);
    }
  };
  // Every softmax and converter warp comes here once its loop has ended: true when all of them may read O^T and the
  // reciprocal row sums.
  auto all_done = [&](bool ok) -> bool {
    if (ok && nt > 0) ok = tc::warp_wait(&bars->odone, (nt - 1) & 1, abort);
    ok = !tc::named_bar_or(2, 32 * (kSoft + kConv), !ok || *abort);
    if (ok) tc::fence_after_sync();
    return ok;
  };

  if (warp < 4) {
    // ------------------------------ MMA issuer ------------------------------
    tc::setmaxnreg_dec<24>();
    if (warp == 0 && nt > 0) {
      const bool lead = tc::elect_one();
      if (lead) {
        tc::mbar_arrive_expect_tx(&bars->qfull, kQBytes);
        for (int ch = 0; ch < 8; ++ch)
          tc::tma_load_3d(base + kOffQ + ch * kQChunk, &tm_q, &bars->qfull, ch * 64, PACK ? q0 * p.H : h0,
                          PACK ? 0 : q0);
      }
      __syncwarp();
      constexpr uint32_t id_qk = tc::idesc_bf16_f32(kRowsT, kHT, false, false);
      constexpr uint32_t id_pv = tc::idesc_bf16_f32(128, kHT, true, true);
      constexpr uint32_t id_pv2 = tc::idesc_bf16_f32(128, 2 * kHT, true, true);  // B = [P_hi | P_lo]
      const uint64_t q_desc0 = tc::sdesc_sw128(tc::smem_u32(base + kOffQ), 16, 1024);
      const uint64_t k_desc0 = tc::sdesc_sw128(tc::smem_u32(base + kOffKv), 16, 1024);
      const uint64_t v_desc0 = tc::sdesc_sw128(tc::smem_u32(base + kOffKv), kKvChunk, 1024);
      const uint64_t p_desc0 = tc::sdesc_sw128(tc::smem_u32(base + kOffP), kPBytes, 1024);
      bool ok = tc::warp_wait(&bars->qfull, 0, abort);
      for (int i = 0; ok && i < nt; ++i) {
        const uint32_t ph = i & 1;
        // S(i-1) has been read: P(i-1), which PV(i-1) waited for, was written after
#pragma unroll 1
        for (int b = 0; b < kBlocks; ++b) {
          if (!(ok = tc::warp_wait(&bars->vfull[b], ph, abort))) break;
          tc::fence_after_sync();
          const uint64_t kd = k_desc0 + b * (2 * kKvChunk >> 4), qd = q_desc0 + b * (2 * kQChunk >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_bf16_lead(lead, tmem + kColS, kd + 2 * k, qd + 2 * k, id_qk, b + k > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_bf16_lead(lead, tmem + kColS, kd + (kKvChunk >> 4) + 2 * k, qd + (kQChunk >> 4) + 2 * k, id_qk, 1u);
        }
        if (!ok) break;
        if (lead) tc::mma_commit(&bars->sfull);
        __syncwarp();
        if (!(ok = tc::warp_wait(&bars->pfull, ph, abort))) break;
        tc::fence_after_sync();
#pragma unroll 1
        for (int b = 0; b < kBlocks; ++b) {
          const uint64_t vd = v_desc0 + b * (2 * kKvChunk >> 4);
          const uint32_t od = tmem + kColO + b * kColBlock;
          if (b < kBlocks - 1) {
#pragma unroll
            for (int kk = 0; kk < kRowsT / 16; ++kk)  // (the columns of P_lo are the operand's next 64)
              tc::mma_bf16_lead(lead, od, vd + kk * (2048 >> 4), p_desc0 + kk * (2048 >> 4), id_pv2,
                                i + kk > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < kRowsT / 16; ++kk) {
              tc::mma_bf16_lead(lead, od, vd + kk * (2048 >> 4), p_desc0 + kk * (2048 >> 4), id_pv,
                                i + kk > 0 ? 1u : 0u);
              tc::mma_bf16_lead(lead, od, vd + kk * (2048 >> 4), p_desc0 + ((kPBytes + kk * 2048) >> 4), id_pv, 1u);
            }
          }
          if (lead) tc::mma_commit(&bars->vempty[b]);  // the converters may refill this block
          __syncwarp();
        }
        if (lead) tc::mma_commit(&bars->odone);
        __syncwarp();
      }
      if (lead) {
        tc::mma_commit(&bars->drain);
        for (uint32_t k = 0; k < tc::kSpinLimit && !tc::mbar_try_wait(&bars->drain, 0); ++k) __nanosleep(64);
        for (uint32_t k = 0; k < tc::kSpinLimit && !tc::mbar_try_wait(&bars->qfull, 0); ++k) __nanosleep(64);
      }
    }
  } else if (warp < 4 + kSoft) {
    // ------------------------------ softmax ------------------------------
    tc::setmaxnreg_dec<64>();
    const int hsel = (warp - 4) >> 2;  // columns [32 hsel, 32 hsel + 32)
    const int row = quarter * 32 + lane, st = threadIdx.x - 128;
    const float scale_log2 = p.scale * kLog2e;
    // The rotation by -t of the output channels that this thread will hold in the last two blocks (unsplit queries):
    // taken now, while the first rows are under way.  Channel d pairs with d ^ 1, the neighbouring lane.
    float rc0 = 1.f, rs0 = 0.f, rc1 = 1.f, rs1 = 0.f;
    if (!PACK && splits == 1 && p.rope_dims > 0) {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const int d = (kBlocks - 2 + k) * 128 + row - (kC - p.rope_dims);
        float cs = 1.f, sn = 0.f;
        if (d >= 0) rope_cos_sin(grp.t, d >> 1, p.rope_dims, p.rope_base, cs, sn);
        rc0 = rc1;
        rs0 = rs1;
        rc1 = cs;
        rs1 = (d & 1) ? -sn : sn;
      }
    }
    // Columns are taken 16 at a time, to keep the registers of a thread few.
    float lw = 0.f;  // lane l: column 32 hsel + l's sum over this warp's rows, relative to the running maximum
    unsigned char* prow = base + kOffP + row * 128;
    // 128-byte part of this row of the tile in chunk ch.
    auto row_part = [&](int ch) -> uint4* {
      return reinterpret_cast<uint4*>(base + kOffKv + ch * kKvChunk + row * 128);
    };
    bool failed = false;
    int i = 0, g = 0;
    for (int j = 0; j < grp.n && !failed;) {
      const Run r = grp.run(p, j, lane);
      j = r.j1;
      const int la = max(ga - g, 0), lb = min(gb - g, r.n);
      g += r.n;
      // packed: the rows that column 32 hsel + lane sees: entries below ecount; window tokens wlo .. wlo + wcount - 1
      int ecount = 0, wlo = 0, wcount = 0;
      if (PACK) {
        const int jc = (32 * hsel + lane) / p.H;
        const int tj = __shfl_sync(0xffffffffu, grp.t, min(jc, 31)), vj = __shfl_sync(0xffffffffu, grp.vis, min(jc, 31));
        if (jc >= r.j0 && jc < r.j1) {
          ecount = vj;
          wlo = max(0, tj - p.n_win + 1);
          wcount = tj - wlo + 1;
        }
      }
      for (int lt = la; lt < lb; ++lt, ++i) {
        const uint32_t ph = i & 1;
        // (block 0 landed long before S: this wait orders the converters' row flags before their use here)
        failed = !tc::warp_wait(&bars->vfull[0], ph, abort) || !tc::warp_wait(&bars->sfull, ph, abort);
        const bool valid = !failed && ((bars->rowok[i & 3][row >> 3] >> (4 * (row & 7))) & 1u);
        const uint32_t vmask = valid ? 0xffffffffu : 0u;
        // Columns that see this row.  Only tiles with rows that some column of the group does not see look at them.
        uint32_t sees = 0xffffffffu;
        const bool masked = PACK && (r.j1 - r.j0 < grp.n || lt >= r.na || (lt + 1) * kRowsT > r.least);
        if (masked) {
          const uint32_t pos = lt < r.na ? lt * kRowsT + row : (uint32_t)r.tok0 + (lt - r.na) * kRowsT + row;
          sees = 0u;
#pragma unroll 1
          for (int c = 0; c < 32; ++c) {
            const int lo = __shfl_sync(0xffffffffu, lt < r.na ? 0 : wlo, c);
            const int n = __shfl_sync(0xffffffffu, lt < r.na ? ecount : wcount, c);
            if (pos - (uint32_t)lo < (uint32_t)n) sees |= 1u << c;
          }
        }
        // A row with an infinity or a NaN that only some columns see must not reach the others as 0 * NaN: it is zeroed
        // for PV, and the columns that see it get a NaN weight.  Its score is not finite in any column, so one tells
        // where to look.  (S has been formed: QK^T does not read the row again.)
        bool nonfinite = false;
        if (PACK && masked) {
          if (!failed) tc::fence_after_sync();
          uint32_t s0 = 0u;
          if (!failed) {
            tc::tmem_ld1(tmem + lanebase + kColS + kHpt * hsel, s0);
            tc::tmem_ld_wait();
          }
          const bool odd = valid && (s0 & 0x7f800000u) == 0x7f800000u;
          if (tc::named_bar_or(1, 32 * kSoft, odd)) {
            if (odd) {
#pragma unroll 1
              for (int w = 0; w < 64; ++w) nonfinite |= any_not_finite(row_part(w >> 3)[w & 7]);
            }
            tc::named_bar(1, 32 * kSoft);  // (both warps of the quarter have looked)
            if (nonfinite) {
#pragma unroll 1
              for (int w = 32 * hsel; w < 32 * hsel + 32; ++w) row_part(w >> 3)[w & 7] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        // scores of heads 16 x .. 16 x + 15 of this warp's
        auto load_scores = [&](int x, uint32_t (&v)[16]) {
          tc::tmem_ld16(tmem + lanebase + kColS + kHpt * hsel + 16 * x, v);
          tc::tmem_ld_wait();
        };
        // P(i) against the running maxima (PV(i-1), the last reader of the buffer, has completed), zeros in rows that
        // take no part; returns the largest score (in units of log2) relative to its head's maximum.  The first pass takes
        // references below kLarge for granted.
        auto write_p = [&](auto first_pass) -> float {
          float top = neg_inf();
#pragma unroll
          for (int x = 0; x < kHpt / 16; ++x) {
            uint32_t v[16], w[8];
            load_scores(x, v);
            float sv[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float4 m4 = *reinterpret_cast<const float4*>(bars->nref + kHpt * hsel + 16 * x + 4 * c);
              sv[4 * c] = fmaf(__uint_as_float(v[4 * c]), scale_log2, m4.x);
              sv[4 * c + 1] = fmaf(__uint_as_float(v[4 * c + 1]), scale_log2, m4.y);
              sv[4 * c + 2] = fmaf(__uint_as_float(v[4 * c + 2]), scale_log2, m4.z);
              sv[4 * c + 3] = fmaf(__uint_as_float(v[4 * c + 3]), scale_log2, m4.w);
            }
            if constexpr (!decltype(first_pass)::value) {
#pragma unroll
              for (int h = 0; h < 16; ++h) {
                const float m = bars->nref[kHpt * hsel + 16 * x + h];
                if (fabsf(m) >= kLarge) sv[h] = __fadd_rn(__fmul_rd(__uint_as_float(v[h]), scale_log2), m);
              }
            }
            if (PACK && masked) {
#pragma unroll
              for (int h = 0; h < 16; ++h)
                sv[h] = (sees >> (16 * x + h)) & 1u ? (nonfinite ? __uint_as_float(0x7fffffffu) : sv[h]) : neg_inf();
            }
#pragma unroll
            for (int h = 0; h < 16; h += 2) top = fmaxf(top, fmaxf(sv[h], sv[h + 1]));
            uint32_t wl[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float p0 = fast_exp2(sv[2 * k]), p1 = fast_exp2(sv[2 * k + 1]);
              const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
              w[k] = prmt_raw(u0, u1, 0x7632u) & vmask;
              wl[k] = pack_bf16x2(p0 - __uint_as_float(u0 & 0xffff0000u), p1 - __uint_as_float(u1 & 0xffff0000u)) & vmask;
            }
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              const int c = (kHpt / 8) * hsel + 2 * x + cc;  // 16-byte unit of the row: columns 8c .. 8c+7
              unsigned char* to = prow + ((c ^ (row & 7)) << 4);
              *reinterpret_cast<uint4*>(to) = make_uint4(w[4 * cc], w[4 * cc + 1], w[4 * cc + 2], w[4 * cc + 3]);
              *reinterpret_cast<uint4*>(to + kPBytes) =
                  make_uint4(wl[4 * cc], wl[4 * cc + 1], wl[4 * cc + 2], wl[4 * cc + 3]);
            }
          }
          return valid ? top : neg_inf();
        };
        if (!failed) tc::fence_after_sync();
        if (i == 0) {
          // The first row's scores as the first references: none exceeds its column's maximum.
          if (quarter == 0) {
#pragma unroll 1
            for (int x = 0; x < kHpt / 16; ++x) {
              uint32_t v[16];
              load_scores(x, v);
              if (lane == 0 && valid) {
#pragma unroll
                for (int h = 0; h < 16; ++h) {
                  const float m = __fmul_rd(__uint_as_float(v[h]), scale_log2);
                  if (((sees >> (16 * x + h)) & 1u) && fabsf(m) <= -kNoMax) {
                    bars->nref[kHpt * hsel + 16 * x + h] = -m;
                    if (fabsf(m) >= kLarge) bars->large = 1;
                  }
                }
              }
            }
          }
          tc::named_bar(1, 32 * kSoft);
        }
        const float top = write_p(std::true_type{});
        // One vote for "no score lies above its head's running reference + 20, no reference is large and nobody failed", the
        // usual case: P stands.  Otherwise new maxima, rescaled accumulators, and P again.
        if (tc::named_bar_or(1, 32 * kSoft, top > kRescaleLog2 || failed || *abort_or_large != 0)) {
          if (tc::named_bar_or(1, 32 * kSoft, failed || *abort)) { failed = true; break; }
#pragma unroll 1
          for (int x = 0; x < kHpt / 16; ++x) {
            uint32_t v[16];
            load_scores(x, v);
            const uint32_t ok = (sees & vmask) >> (16 * x);
            float m = 0.f;
#pragma unroll
            for (int h = 0; h < 16; ++h) {
              const float y = warp_max((ok >> h) & 1u ? __fmul_rd(__uint_as_float(v[h]), scale_log2) : neg_inf());
              if (lane == h) m = y;
            }
            if (lane < 16) bars->red[quarter][kHpt * hsel + 16 * x + lane] = m;
          }
          tc::named_bar(1, 32 * kSoft);
          if (st < kHT) {
            const float mt = fmaxf(fmaxf(bars->red[0][st], bars->red[1][st]), fmaxf(bars->red[2][st], bars->red[3][st]));
            const float mo = -bars->nref[st];
            const bool grow = mt > mo + kRescaleLog2;
            bars->alpha[st] = grow ? fast_exp2(mo - mt) : 1.f;
            if (grow) {
              bars->nref[st] = -mt;
              if (fabsf(mt) >= kLarge) bars->large = 1;
            }
          }
          tc::named_bar(1, 32 * kSoft);
          lw *= bars->alpha[kHpt * hsel + lane];
          if (i > 0) {
            // O^T holds the sums up to tile i-1 (PV(i-1) was issued before QK(i), whose commit has arrived)
            tc::fence_after_sync();
#pragma unroll 1
            for (int part = 0; part < (2 * kBlocks - 1) * (kHpt / 16); ++part) {
              const int hh = kHpt * hsel + 16 * (part & 1);
              const uint32_t ta = tmem + lanebase + kColO + (part >> 1) * kHT + hh;  // (64 columns of a term each)
              uint32_t v[16];
              tc::tmem_ld16(ta, v);
              tc::tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < 16; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) * bars->alpha[hh + h]);
              tc::tmem_st16(ta, v);
            }
            tc::tmem_st_wait();
          }
          write_p(std::false_type{});
        }
        tc::fence_before_sync();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->pfull);
        // the row sums of exactly what PV multiplies, read back from this thread's own row
#pragma unroll 1
        for (int x = 0; x < kHpt / 16; ++x) {
          float sv[16];
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int c = (kHpt / 8) * hsel + 2 * x + cc;
            const unsigned char* at = prow + ((c ^ (row & 7)) << 4);
            float f[8], lo[8];
            unpack8(*reinterpret_cast<const uint4*>(at), f);
            unpack8(*reinterpret_cast<const uint4*>(at + kPBytes), lo);
#pragma unroll
            for (int h = 0; h < 8; ++h) sv[8 * cc + h] = f[h] + lo[h];
          }
          const float t = warp_sum16(sv, lane);
          if ((lane >> 4) == x) lw += t;
        }
      }
    }
    // ---- epilogue: O^T (channels x columns) and the row sums ----
    bars->red[quarter][kHpt * hsel + lane] = lw;
    tc::named_bar(1, 32 * kSoft);
    if (!failed && st < kHT) {
      float l = (bars->red[0][st] + bars->red[1][st]) + (bars->red[2][st] + bars->red[3][st]);
      if (PACK || splits > 1) {
        const int to = column_row(st);
        if (to >= 0) ws_ml[to] = make_float2(l > 0.f ? -bars->nref[st] : neg_inf(), l);
      } else {
        // a sink logit joins the denominator here (base-2, against the running maximum), for partial states in the
        // combine
        if (p.sink != nullptr && h0 + st < p.H && l > 0.f) l += fast_exp2(p.sink[h0 + st] * kLog2e + bars->nref[st]);
        bars->alpha[st] = l == 0.f ? 0.f : __fdividef(1.f, l);  // (NaN stays)
      }
    }
    if (all_done(!failed)) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k)
        store_part(2 + (k >> 1), 2 * hsel + (k & 1), k < 2 ? rc0 : rc1, k < 2 ? rs0 : rs1);
      copy_out();
    }
  } else {
    // ------------------------------ converters ------------------------------
    tc::setmaxnreg_inc<88>();
    const int cw = warp - 4 - kSoft;
    const int row = 8 * cw + (lane >> 2), sub = lane & 3;    // row of the tile; group 4b + sub of block b
    const int n_groups = (kC - p.kv.rope_dims) / kFp4Group;  // groups held in 4 bits
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(p.kv.codes) + sub * 16;
    const uint8_t* scales = reinterpret_cast<const uint8_t*>(p.kv.scales);
    const int chunk = sub >> 1;                              // of a block's two
    const uint32_t sw = row & 7;
    // This thread's 16-byte units of its chunk's row are unit0 ^ w, w = 0 .. 3: with the swizzle, the eight lanes of a
    // store phase (two rows, four groups) hit eight different units.
    const uint32_t unit0 = 4 * (sub & 1) + 2 * chunk;
    unsigned char* kv = base + kOffKv + row * 128;
    bool okw = true;
    int i = 0, g = 0;
    for (int j = 0; j < grp.n && okw;) {
      const Run r = grp.run(p, j, lane);
      j = r.j1;
      const int la = max(ga - g, 0), lb = min(gb - g, r.n), le = min(lb, r.na);
      g += r.n;
      // Entry of this thread's row of the run's tile lt (-1: none), among those of this CTA.
      auto entry_of = [&](int lt) -> int {
        const int u = lt * kRowsT + row;
        if (lt >= le || u >= r.entries) return -1;
        return grp.idx ? grp.idx[u] : u;
      };
      // The block that entry e lies in (paged), loaded but not looked at yet, and its cache row from it.
      auto block_of = [&](int e) -> int {
        if (!p.kv.bt || e < 0 || e >= p.N) return 0;
        const unsigned int j = div_by(e, p.kv.div);
        return j < p.kv.bt_stride ? p.kv.bt[r.req * p.kv.bt_stride + j] : -1;
      };
      auto resolve = [&](int lt, int e, int blk) -> int {
        if (p.check && sub == 0 && grp.idx && lt < le && lt * kRowsT + row < r.entries) {
          const unsigned int k = entry_check(e, grp.t, p.rate, p.N);
          if (k) atomicOr(&g_mqa_fp4_error, k << 1);
        }
        if (e < 0 || e >= p.N) return -1;
        const int in_block = e - (int)(div_by(e, p.kv.div) * p.kv.div.d);
        long long x = p.kv.bt ? (blk < 0 ? -1ll : (long long)blk * p.kv.rpb + in_block)
                              : (e < p.kv.seq_rows ? r.req * p.kv.seq_rows + e : -1ll);
        if (x >= p.kv.n_rows) x = -1;
        if (p.check && x < 0) atomicOr(&g_mqa_fp4_error, kIdxBlock << 1);
        return (int)x;
      };
      // The codes of this thread's group of block b of cache row x, in the order of its stores (halves swapped in the
      // second chunk).
      auto fetch = [&](int x, int b) -> uint4 {
        const uint4 v = x >= 0 && 4 * b + sub < n_groups
                            ? *reinterpret_cast<const uint4*>(codes + x * p.kv.ld_codes + b * 64)
                            : make_uint4(0u, 0u, 0u, 0u);
        return chunk ? make_uint4(v.z, v.w, v.x, v.y) : v;
      };
      auto fetch_scales = [&](int x) -> uint4 {
        return x >= 0 ? *reinterpret_cast<const uint4*>(scales + x * p.kv.ld_scales) : make_uint4(0u, 0u, 0u, 0u);
      };
      // Copies a quarter of a 128-byte row of chunk c (units 2 sub and 2 sub + 1); zeros where there is none.
      auto copy_row = [&](int c, const bf16* src, bool ok) {
        const uint32_t dst = tc::smem_u32(kv + c * kKvChunk);
#pragma unroll
        for (uint32_t w = 0; w < 2; ++w)
          tc::cp_async16(dst + (((2 * sub + w) ^ sw) << 4), src + (2 * sub + w) * 8, ok ? 16 : 0);
      };
      // The rotary channels of cache row x on their way to L2.
      auto fetch_rope = [&](int x) {
        if (x >= 0 && sub == 0 && p.kv.rope_dims > 0)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.kv.rope + x * p.kv.ld_rope));
      };
      // An entry's index, its block and its row are dependent loads, each given a tile's time: x is the cache row of the
      // tile being converted, e1 and b1 entry and block of the next one, e2 the entry of the one after.
      const int e0 = entry_of(la);
      int e1 = entry_of(la + 1), e2 = entry_of(la + 2);
      int x = resolve(la, e0, block_of(e0));
      int b1 = block_of(e1);
      fetch_rope(x);
      // This thread's group of block b in bf16, in the order of its stores: widened, or rotary channels as they are.
      auto widen = [&](int b, const uint4& v, uint32_t scale_word, uint4 (&o)[4]) {
        const int g = 4 * b + sub;
        if (g < n_groups) {
          e2m1x32_to_bf16(v, (scale_word >> (8 * sub)) & 255u, o);
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(p.kv.rope + (x >= 0 ? x * p.kv.ld_rope : 0ll) +
                                                            (g - n_groups) * 32);
#pragma unroll
          for (int w = 0; w < 4; ++w) o[w] = x >= 0 ? src[(2 * chunk) ^ w] : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      // Store such a group and signal the block.
      auto put = [&](int b, const uint4 (&o)[4]) {
        unsigned char* d = kv + (2 * b + chunk) * kKvChunk;
#pragma unroll
        for (uint32_t w = 0; w < 4; ++w) *reinterpret_cast<uint4*>(d + (((unit0 ^ w) ^ sw) << 4)) = o[w];
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->vfull[b]);
      };
      int lt = la;
      for (; okw && lt < le; ++lt, ++i) {
        const uint32_t ph = i & 1;
        const uint32_t mask = __ballot_sync(0xffffffffu, x >= 0);
        if (lane == 0) bars->rowok[i & 3][cw] = mask;
        uint4 oa[4], ob[4], oc[4];
        const uint4 sc = fetch_scales(x);
        const uint4 v0 = fetch(x, 0), v1 = fetch(x, 1), v2 = fetch(x, 2), v3 = fetch(x, 3);
        widen(0, v0, sc.x, oa);
        widen(1, v1, sc.y, ob);
        widen(2, v2, sc.z, oc);
        if (!(okw = tc::warp_wait(&bars->vempty[0], ph ^ 1, abort))) break;
        put(0, oa);
        widen(3, v3, sc.w, oa);
        if (!(okw = tc::warp_wait(&bars->vempty[kBlocks - 1], ph ^ 1, abort))) break;
        put(1, ob);
        put(2, oc);
        put(3, oa);
        x = resolve(lt + 1, e1, b1);
        fetch_rope(x);
        e1 = e2;
        b1 = block_of(e1);
        e2 = entry_of(lt + 3);
      }
      for (; okw && lt < lb; ++lt, ++i) {  // window rows
        const uint32_t ph = i & 1;
        const int w = (lt - r.na) * kRowsT + row;
        const bool valid = w < r.window;
        const uint32_t mask = __ballot_sync(0xffffffffu, valid);
        if (lane == 0) bars->rowok[i & 3][cw] = mask;
        const bf16* src = valid ? p.win + r.req * p.win_seq_stride + (long long)((r.tok0 + w) % p.win_rows) * kC : p.win;
#pragma unroll 1
        for (int b = 0; b < kBlocks; ++b) {
          if (!tc::warp_wait(&bars->vempty[b], ph ^ 1, abort)) { okw = false; break; }
          copy_row(2 * b, src + b * 128, valid);
          copy_row(2 * b + 1, src + b * 128 + 64, valid);
          tc::cp_async_commit();
          if (b > 0) {
            tc::cp_async_wait<1>();
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars->vfull[b - 1]);
          }
        }
        tc::cp_async_wait<0>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (okw && lane == 0) tc::mbar_arrive(&bars->vfull[kBlocks - 1]);
      }
    }
    tc::cp_async_wait<0>();
    if (all_done(okw)) {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) store_part(k, cw >> 2, 1.f, 0.f);
      copy_out();
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (threadIdx.x == 0 && bars->abort) atomicOr(&g_mqa_fp4_error, 1u);
  if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
}
}  // namespace

extern cudaError_t make_tmap_bf16(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims,
                                  const uint64_t* strides_bytes, uint32_t box_rows);

// Queries that share a CTA's 64 columns (1: none do): as many as there are heads' columns for, but no more than a request
// has queries on average, or a CTA would walk the rows of several requests one after the other.  32 requests of one query
// each at 8 heads, 1,024 entries: 25 us with one query a CTA, 59 us with eight (measured with P as one term); 192 queries
// of one request at 16 heads: 58 us with four a CTA, 108 us with two.  A power of two or the most that fit, so that few
// numbers bound the workspace.
int mqa_fp4_pack(int c, int H, int Tq, long long n_req) {
  if (c != kC || H > kHT / 2) return 1;
  const int most = min(32, kHT / H);
  const long long each = Tq / max(1ll, n_req);
  if (each >= most) return most;
  int pack = 1;
  while (2 * pack <= each) pack *= 2;
  return pack;
}

// Splits per query: fewest tiles on the critical path over whole waves of CTAs (one per SM), a CTA's set-up and
// epilogue counted as three quarters of a tile each (tcgen05); about eight CTAs per SM (CUDA cores).
MqaPlan plan_mqa_fp4(const MqaFp4Problem& p, int num_sms) {
  MqaPlan pl;
  const int entries = p.idx ? p.n_idx : p.N, window = p.win ? p.n_win : 0;
  pl.max_rows = max(1, entries + window);
  const size_t state = (size_t)p.Tq * p.H * ((size_t)p.kv.c * sizeof(float) + sizeof(float2));
  if (p.kv.c == kC) {
    const int pack = p.pack;
    const int tiles = max(1, (entries + kRowsT - 1) / kRowsT + (window + pack - 1 + kRowsT - 1) / kRowsT);
    const long long ctas1 = (long long)((max(1, p.Tq) + pack - 1) / pack) * ((p.H + kHT - 1) / kHT);
    const int smax = (int)min((long long)min(tiles, 1024), max(1ll, 2ll * num_sms / ctas1));
    int best = 1;
    long long best_cost = -1;
    // the fewest splits of each number of tiles per CTA
    for (int s = 1, tpc; s <= smax; s = tpc > 1 ? (tiles + tpc - 2) / (tpc - 1) : smax + 1) {
      tpc = (tiles + s - 1) / s;
      const int eff = (tiles + tpc - 1) / tpc;
      const long long waves = (ctas1 * eff + num_sms - 1) / num_sms;
      const long long cost = waves * (tpc * 4 + 6) + (eff > 1 ? 4 : 0);
      if (best_cost < 0 || cost < best_cost) { best_cost = cost; best = eff; }
    }
    pl.splits = best;
    pl.rows_per_split = 0;  // (tiles are dealt out on the device)
    pl.ws_bytes = best > 1 || pack > 1 ? state * best : 0;
    return pl;
  }
  const int groups = (p.H + kSH - 1) / kSH;
  int splits = (int)max(1ll, (8ll * num_sms) / max(1ll, (long long)p.Tq * groups));
  splits = min(min(splits, 64), (pl.max_rows + kSRows - 1) / kSRows);
  pl.rows_per_split = ((pl.max_rows + splits - 1) / splits + kSRows - 1) / kSRows * kSRows;
  pl.splits = (pl.max_rows + pl.rows_per_split - 1) / pl.rows_per_split;
  pl.ws_bytes = state * pl.splits;
  return pl;
}

template <bool PACK>
static cudaError_t launch_tc(const MqaFp4Problem& p, int pack, int splits, float* ws_o, float2* ws_ml,
                             cudaStream_t stream) {
  // rows of the queries: the heads of one query, those past n_heads read as zeros; packed, the heads of all queries
  CUtensorMap tm_q;
  const uint64_t rows = PACK ? (uint64_t)p.Tq * p.H : (uint64_t)p.H;
  const uint64_t qd[3] = {(uint64_t)kC, rows, PACK ? 1ull : (uint64_t)p.Tq};
  const uint64_t qs[2] = {(uint64_t)kC * 2, rows * kC * 2};
  cudaError_t e = make_tmap_bf16(&tm_q, p.q, 3, qd, qs, kHT);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute((const void*)mqa_fp4_tc_kernel<PACK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  const long long ctas = (long long)((p.Tq + pack - 1) / pack) * (PACK ? 1 : (p.H + kHT - 1) / kHT) * splits;
  mqa_fp4_tc_kernel<PACK><<<(unsigned)ctas, kThreads, kSmemBytes, stream>>>(tm_q, p, pack, splits, ws_o, ws_ml);
  return cudaGetLastError();
}

cudaError_t launch_mqa_fp4(const MqaFp4Problem& p, const MqaPlan& pl, void* ws, cudaStream_t stream, bool pdl) {
  if (p.Tq == 0) return cudaSuccess;
  float* ws_o = reinterpret_cast<float*>(ws);
  float2* ws_ml = reinterpret_cast<float2*>(ws_o + (size_t)p.Tq * pl.splits * p.H * p.kv.c);
  cudaError_t e;
  const int pack = p.pack;
  if (p.kv.c == kC) {
    e = pack > 1 ? launch_tc<true>(p, pack, pl.splits, ws_o, ws_ml, stream)
                 : launch_tc<false>(p, pack, pl.splits, ws_o, ws_ml, stream);
  } else {
    const int groups = (p.H + kSH - 1) / kSH;
    mqa_fp4_simple_kernel<<<(unsigned)(p.Tq * groups * pl.splits), kSThreads, 0, stream>>>(
        p, pl.splits, pl.rows_per_split, ws_o, ws_ml);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  ++g_launch_counter;
  if (p.kv.c == kC && pack == 1 && pl.splits == 1) return cudaSuccess;
  return launch_mqa_combine(ws_o, ws_ml, p.Tq, pl.splits, p.H, p.kv.c, p.out, p.sink, p.q_pos, p.rope_dims, p.rope_base,
                            stream, pdl);
}

unsigned int read_and_clear_mqa_fp4_error() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_mqa_fp4_error, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (v) cudaMemcpyToSymbol(g_mqa_fp4_error, &zero, sizeof(zero));
  return v;
}

}  // namespace hca
