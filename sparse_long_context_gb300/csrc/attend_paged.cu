// Decode attention over a paged cache: the pages of a sequence lie anywhere in a pool
// [N, Hkv, P, D] and are found through its table.
//
// The G query heads of a KV head share every byte read.  A row's tokens are taken in
// units of 16 SG positions (of the context in order, or of the listed pages); the rows' units,
// concatenated, are cut into one nearly equal range per CTA (one CTA per SM), so that rows of
// uneven length fill the GPU, and the last CTA to finish a shared row merges its partials in CTA
// order.  Where few or short rows make that faster, a cluster of CTAs takes a row and merges through
// distributed shared memory.
//
// A unit is streamed by one warp through its own ring of shared-memory stages (tensor-map boxes of
// 16 rows, whose row numbers come from the table), so a late copy holds up one warp only.
// Scores, statistics and sums are fp32.
//
// Bound by memory on long contexts, wherever their pages lie: 32 contexts of 49k to 64k tokens, 2 KV
// heads of 6 query heads and 128 channels in bf16, 279 to 282 us for 1884 MB (6.7 TB/s, the measured copy rate).
// Twelve warps of two stages fill the shared memory: 8 of three take 285 us, 6 of four 291, 6 of two
// with 32 tokens each 282.  In fp32 instructions come next: seven contexts of 1 to 20000 tokens, 8 heads of 8 query heads and
// 64 channels 51 us for 268 MB (floor 40).  Short rows are a chain of latencies (lengths, table, copies,
// merge): 5.2 us for 1000 tokens of 4 heads, 16.8 for 64 lists of 128 pages (floor 10); in ranges the
// prologue takes 3 us and the merge through global memory 3.7, so that 64 uneven rows of up to 4k tokens take 18 us with
// two CTAs a row (floor 10) and 21.5 in ranges.  (Times of the device alone, calls replayed from a graph.)
#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "attend_common.cuh"
#include "launch.h"
#include "mma.cuh"
#include "paged.cuh"
#include "tma.cuh"

namespace sls {

constexpr int kPgMaxGrid = 256;    // CTAs whose ranges are kept in shared memory
constexpr int kPgMaxCluster = 16;
constexpr int kPgMaxRows = 4096;   // rows whose first units are kept there
// The arrival counters' place in a workspace, whatever the shape: no call's partials lie
// where another one's counters are.
constexpr size_t kPgTicketBytes = kPgMaxRows * sizeof(int32_t);
constexpr int kPgMinUnits = 4;     // least units of a CTA in ranges: a shorter job uses fewer CTAs
// Work of a row change (drain, merge, partial and refill) in tokens: 512, 1024 and 2048 took 53.3,
// 53.0 and 56.6 us on the uneven fp32 rows above.
constexpr int kPgSegCost = 1024;
// Rows are not cut (and not merged) where that costs the longest range less than this many ns of work: 64 rows of 1000
// tokens 15.7 -> 13.3 us, 128 of 2000 32.0 -> 27.8, 256 of up to 500 21.6 -> 17.0, 64 of 100 11.2 -> 8.4 (5000 ns: 128
// rows of up to 2000 tokens 24.0 for 21.2; moving every border that is within 4 us of a row's start: 64 of up to 4096
// tokens 23.2 for 21.5).
constexpr double kPgWhole = 7000;

struct PagedAttend {
  const void* q;
  const int32_t *table, *page_idx, *count, *ctx_len;
  int idx_stride, k_fixed, rows, Hq, Hkv, G, Cap, P, pshift, pool, test_wait, cluster;
  float qscale;  // softmax scale * log2(e)
  const float* sink;
  void* out;
  float* lse;
  int32_t* tickets;     // [rows] arrival counters, zero between calls
  float *po, *pm, *pl;  // [slot][G][D], [slot][G] partials, two slots per CTA, max in base-2 units
};

__device__ __forceinline__ float pg_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory offset of 16-byte chunk c of row t of a box of 128-byte rows under the copy
// engine's 128-byte swizzle; pieces of 16 rows follow each other.
__device__ __forceinline__ uint32_t pg_chunk(int t, int c) {
  return ((c >> 3) << 11) + (t << 7) + (((c ^ t) & 7) << 4);
}

// ---- one warp's state and work, by element type

// bf16 on the tensor cores (m16n8k16):
//   S = Q K^T        A = the heads' queries (rows 0-7), B = keys
//   O^T += V^T P^T   A = values (transposed as they are read), B = the weights in a high and a low bf16 part
// A weight's high part is truncated and the low one rounded: 16 bits in all, half a step 2^-15 of the
// weight, so that the output is off by its own rounding only.
template <int D_>
struct PgBf16 {
  using T = bf16;
  static constexpr int D = D_, W = 12, S = 2, SG = D == 128 ? 1 : 2, KS = D / 16;
  static constexpr int GROUP = 16 * D * 2, STAGE = 2 * SG * GROUP;
  static constexpr double NS = D == 128 ? 4.6 : 3.0;  // a token of a CTA by itself
  uint32_t qa[KS][2];
  float o[KS][4], m_run, l_run;  // head lane / 4; accumulator columns are heads 2m and 2m + 1

  __device__ __forceinline__ void start(const T* q, int G, int lane) {
    const int r = lane >> 2, m = lane & 3;
#pragma unroll
    for (int c = 0; c < KS; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        qa[c][i] = r < G ? ld_global(reinterpret_cast<const uint32_t*>(q + r * D + 16 * c + 8 * i + 2 * m)) : 0u;
#pragma unroll
    for (int t = 0; t < KS; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    m_run = kNegInf;
    l_run = 0.f;
  }

  // A unit in `stage`: group s has lim[s] valid tokens.
  __device__ __forceinline__ void unit(uint32_t stage, const int (&lim)[SG], float qscale, int lane) {
    const int m = lane & 3, j = lane >> 3, row = 8 * (j >> 1) + (lane & 7);
    float x[SG][4], gm = kNegInf;
#pragma unroll
    for (int s = 0; s < SG; ++s) {
      float sc[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[0][i] = sc[1][i] = 0.f;
      if (lim[s] > 0) {
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          uint32_t w[4];
          ldsm_x4(stage + s * GROUP + pg_chunk(row, 2 * c + (j & 1)), w[0], w[1], w[2], w[3]);
          mma_bf16(sc[0], qa[c][0], 0u, qa[c][1], 0u, w[0], w[1]);
          mma_bf16(sc[1], qa[c][0], 0u, qa[c][1], 0u, w[2], w[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 2 * m + (i & 1) + 8 * (i >> 1);
        x[s][i] = t < lim[s] ? sc[i >> 1][i & 1] * qscale : kNegInf;
        gm = fmaxf(gm, x[s][i]);
      }
    }
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
    const float mn = fmaxf(m_run, gm), mref = mn == kNegInf ? 0.f : mn;
    const float alpha = pg_ex2(m_run - mref);  // before any token: exp2(-inf) = 0 scales zeros
    m_run = mn;
    l_run *= alpha;
    const float a_lo = __shfl_sync(0xffffffffu, alpha, 8 * m), a_hi = __shfl_sync(0xffffffffu, alpha, 8 * m + 4);
    if (!__all_sync(0xffffffffu, a_lo == 1.f && a_hi == 1.f)) {
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        o[t][0] *= a_lo; o[t][1] *= a_hi; o[t][2] *= a_lo; o[t][3] *= a_hi;
      }
    }
#pragma unroll
    for (int s = 0; s < SG; ++s) {
      if (lim[s] <= 0) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[s][i] = pg_ex2(x[s][i] - mref);
      l_run += (x[s][0] + x[s][1]) + (x[s][2] + x[s][3]);
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        hi[i] = __byte_perm(__float_as_uint(x[s][2 * i]), __float_as_uint(x[s][2 * i + 1]), 0x7632);
        lo[i] = pack_bf16(x[s][2 * i] - bf16lo(hi[i]), x[s][2 * i + 1] - bf16hi(hi[i]));
        // a low part of zero becomes 2^-126 next to a weight: an infinite value meets no zero
        lo[i] = __vmaxu2(lo[i], 0x00800080u) & __vcmpgtu2(hi[i], 0u);
      }
      const uint32_t v = stage + (SG + s) * GROUP;
      if (lim[s] >= 16) {
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4_t(v + pg_chunk(row, 2 * t + (j & 1)), a0, a1, a2, a3);
          mma_bf16(o[t], a0, a1, a2, a3, hi[0], hi[1]);
          mma_bf16(o[t], a0, a1, a2, a3, lo[0], lo[1]);
        }
      } else {  // rows behind the context count as zero, whatever they hold
        uint32_t keep[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          keep[i] = (2 * m + 8 * i < lim[s] ? 0xffffu : 0u) | (2 * m + 8 * i + 1 < lim[s] ? 0xffff0000u : 0u);
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4_t(v + pg_chunk(row, 2 * t + (j & 1)), a0, a1, a2, a3);
          a0 &= keep[0]; a1 &= keep[0]; a2 &= keep[1]; a3 &= keep[1];
          mma_bf16(o[t], a0, a1, a2, a3, hi[0], hi[1]);
          mma_bf16(o[t], a0, a1, a2, a3, lo[0], lo[1]);
        }
      }
    }
  }

  // sO [head][D + 4], sM, sL [head] of this warp
  __device__ __forceinline__ void finish(float* sO, float* sM, float* sL, bool ok, int lane) {
    const int r = lane >> 2, m = lane & 3;
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
    if (m == 0) {
      sM[r] = ok ? m_run : __int_as_float(0x7f800000);
      sL[r] = l_run;
    }
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      float* p = sO + 2 * m * (D + 4) + 16 * t + r;
      p[0] = o[t][0];
      p[D + 4] = o[t][1];
      p[8] = o[t][2];
      p[D + 12] = o[t][3];
    }
  }
};

// Two floats in one 64-bit register: products and sums of both at once.
using PgF2 = unsigned long long;
__device__ __forceinline__ PgF2 pg_f2(float lo, float hi) {
  PgF2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 pg_split(PgF2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ PgF2 pg_fma(PgF2 a, PgF2 b, PgF2 c) {
  PgF2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ PgF2 pg_mul(PgF2 a, PgF2 b) {
  PgF2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void pg_lds(uint32_t at, PgF2& a, PgF2& b) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(at));
}
__device__ __forceinline__ void pg_lds(uint32_t at, PgF2& a) {
  asm volatile("ld.shared.u64 %0, [%1];" : "=l"(a) : "r"(at));
}

// fp32 on the CUDA cores, no operand rounded.  Scores: lane (tg, sl) takes channel chunks sl, sl + 8, ... of tokens
// 4 j + tg, with the heads' queries in registers; the eight lanes of a token add up so that lane sl ends with head
// sl.  The weights go to shared memory twice each (over the unit's keys, which are done with), as the pairs that the
// value product multiplies a lane's D / 32 channels by.  12 warps at D = 64: 11, 10 and 8 (three stages) took 55, 60
// and 56 us for 53.  GM: heads that are worked on (4 or 8; a check of each
// against G would cost as many instructions as its products).
template <int D_, int GM>
struct PgF32 {
  using T = float;
  static constexpr int D = D_, W = D == 128 ? 6 : 12, S = 2, SG = 1;
  static constexpr int GROUP = 16 * D * 4, STAGE = 2 * GROUP, NF = D / 64, NC = D / 32;
  static constexpr double NS = D == 128 ? 19.0 : 8.3;  // a token of a CTA by itself
  PgF2 q[GM][NC][2], o[GM][NF];
  float m_run, l_run;  // of head sl % GM; the sum of this lane's tokens

  __device__ __forceinline__ void start(const T* qp, int G, int lane) {
    const int sl = lane & 7;
#pragma unroll
    for (int g = 0; g < GM; ++g) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int h = g ^ (sl & (GM - 1));  // so that what a lane keeps when the lanes add up has fixed places
        const float4 v = h < G ? ld_global(reinterpret_cast<const float4*>(qp + h * D + 32 * i + 4 * sl))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
        q[g][i][0] = pg_f2(v.x, v.y);
        q[g][i][1] = pg_f2(v.z, v.w);
      }
#pragma unroll
      for (int i = 0; i < NF; ++i) o[g][i] = 0ull;
    }
    m_run = kNegInf;
    l_run = 0.f;
  }

  __device__ __forceinline__ void unit(uint32_t stage, const int (&lims)[1], float qscale, int lane) {
    const int tg = lane >> 3, sl = lane & 7, lim = lims[0];
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      PgF2 k[NC][2];
#pragma unroll
      for (int i = 0; i < NC; ++i) pg_lds(stage + pg_chunk(4 * j + tg, 8 * i + sl), k[i][0], k[i][1]);
      float s[GM];
#pragma unroll
      for (int g = 0; g < GM; ++g) {
        PgF2 a = pg_mul(q[g][0][0], k[0][0]);
        a = pg_fma(q[g][0][1], k[0][1], a);
#pragma unroll
        for (int i = 1; i < NC; ++i) a = pg_fma(q[g][i][1], k[i][1], pg_fma(q[g][i][0], k[i][0], a));
        const float2 d = pg_split(a);
        s[g] = d.x + d.y;
      }
      // the heads over the eight lanes (place g of lane sl is head g ^ sl): half of what is left goes to the other
      // half of the lanes
      if constexpr (GM == 4)
#pragma unroll
        for (int g = 0; g < 4; ++g) s[g] += __shfl_xor_sync(0xffffffffu, s[g], 4);
#pragma unroll
      for (int w = GM / 2; w > 0; w >>= 1)
#pragma unroll
        for (int g = 0; g < w; ++g) s[g] += __shfl_xor_sync(0xffffffffu, s[g + w], w);
      x[j] = 4 * j + tg < lim ? s[0] * qscale : kNegInf;
    }
    float gm = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 8));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 16));
    const float mn = fmaxf(m_run, gm), mref = mn == kNegInf ? 0.f : mn;
    const float alpha = pg_ex2(m_run - mref);
    m_run = mn;
    if (!__all_sync(0xffffffffu, alpha == 1.f)) {
      l_run *= alpha;
#pragma unroll
      for (int g = 0; g < GM; ++g) {
        const float f = __shfl_sync(0xffffffffu, alpha, g);
#pragma unroll
        for (int i = 0; i < NF; ++i) o[g][i] = pg_mul(o[g][i], pg_f2(f, f));
      }
    }
    __syncwarp();  // every lane has read the keys
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float p = pg_ex2(x[j] - mref);
      l_run += p;
      asm volatile("st.shared.v2.f32 [%0], {%1, %1};" ::"r"(stage + (4 * j + tg) * 8 * GM + sl % GM * 8), "f"(p) : "memory");
    }
    __syncwarp();
    const uint32_t v = stage + GROUP;
    auto token = [&](int t) {
      PgF2 y[NF], p[GM];
      if constexpr (NF == 2) pg_lds(v + pg_chunk(t, lane), y[0], y[1]);
      else pg_lds(v + pg_chunk(t, lane >> 1) + 8 * (lane & 1), y[0]);
#pragma unroll
      for (int g = 0; g < GM; g += 2) pg_lds(stage + t * 8 * GM + g * 8, p[g], p[g + 1]);
#pragma unroll
      for (int g = 0; g < GM; ++g)
#pragma unroll
        for (int i = 0; i < NF; ++i) o[g][i] = pg_fma(y[i], p[g], o[g][i]);
    };
    if (lim >= 16) {
#pragma unroll
      for (int t = 0; t < 16; ++t) token(t);
    } else {  // rows behind the context are not read
#pragma unroll 1
      for (int t = 0; t < lim; ++t) token(t);
    }
  }

  __device__ __forceinline__ void finish(float* sO, float* sM, float* sL, bool ok, int lane) {
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 8);
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 16);
    if (lane < GM) {
      sM[lane] = ok ? m_run : __int_as_float(0x7f800000);
      sL[lane] = l_run;
    }
#pragma unroll
    for (int g = 0; g < GM; ++g)
#pragma unroll
      for (int i = 0; i < NF; ++i)
        *reinterpret_cast<float2*>(sO + g * (D + 4) + lane * 2 * NF + 2 * i) = pg_split(o[g][i]);
  }
};

// ---- the kernel

constexpr int kPgWeights = 160;  // contributors of a row whose weights are kept (all SMs of a GB300)
template <bool CL>
struct PgSmem {
  int s_lo[CL ? 1 : kPgMaxGrid + 1];  // first unit of every CTA's range, and the total
  int s_slot[CL ? 1 : kPgMaxGrid];
  int s_tmp[32];
  int s_fail, s_ncontrib, s_last;
  float s_w[8][CL ? 1 : kPgWeights], s_m[8], s_inv[8];
};

// Final output of head hq, channel d: accumulator av and sum lv relative to exp2(M); the sink joins the sum.
template <typename T, int D>
__device__ __forceinline__ void pg_finish(const PagedAttend& a, size_t hq, int head, float M, float lv, float av, int d) {
  const float sk = a.sink ? a.sink[head] * kLog2e : kNegInf;
  const float Mx = fmaxf(M, sk);
  float f = 0.f, Lt = 0.f;
  if (Mx != kNegInf) {
    f = M == kNegInf ? 0.f : pg_ex2(M - Mx);
    Lt = lv * f + (a.sink ? pg_ex2(sk - Mx) : 0.f);
  }
  // a NaN sum (NaN scores, or a wait that gave up) stays NaN in the output and lse
  static_cast<T*>(a.out)[hq * D + d] = from_f32<T>(Lt == 0.f ? 0.f : av * f / Lt);
  if (d == 0 && a.lse) a.lse[hq] = Lt == 0.f ? kNegInf : Mx * kLn2 + logf(Lt);
}

// What the CTAs of a row's cluster send each other: rank r merges its share of
// the G x D outputs, a multiple of 4 values.
template <int D>
struct __align__(16) PgInbox {
  float o[8 * D + 4 * kPgMaxCluster];
  float m[kPgMaxCluster * 8], l[kPgMaxCluster * 8];
};

template <typename Tile>
struct PgLayout {
  static constexpr size_t RING = (size_t)Tile::W * Tile::S * Tile::STAGE;
  static constexpr int MROW = Tile::D + 4;
  static constexpr size_t MERGE = (size_t)Tile::W * 8 * MROW * sizeof(float);
  static constexpr size_t REGION = RING > MERGE ? RING : MERGE;
  static constexpr size_t smem(int rows) { return REGION + (size_t)(rows + 1) * sizeof(int) + 1024; }
};

// CL: the CTAs of a cluster take one row's units in equal shares and merge through
// distributed shared memory; otherwise every CTA takes a range of all rows' units.
template <typename Tile, bool LIST, bool CL>
__global__ void __launch_bounds__(Tile::W * 32, 1)
paged_attend_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const PagedAttend a) {
  using L = PgLayout<Tile>;
  using T = typename Tile::T;
  constexpr int D = Tile::D, W = Tile::W, S = Tile::S, SG = Tile::SG, NT = W * 32, UT = 16 * SG;
  constexpr int BATCH = 32 - (S - 1);  // units between two loads of a warp's page numbers
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  int* s_pref = reinterpret_cast<int*>(ring + L::REGION);  // [rows + 1] first unit of each row
  __shared__ PgSmem<CL> sh;
  __shared__ uint64_t full[W][S];
  __shared__ float sM[W][8], sL[W][8], sF[W][8], sHm[8], sHl[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G, rows = a.rows, cta = blockIdx.x, MP = a.Cap >> a.pshift;
  if (threadIdx.x == 0) {
    for (int w = 0; w < W; ++w)
      for (int s = 0; s < S; ++s) mbar_init(&full[w][s], 1);
    mbar_fence_init();
    tma_prefetch_map(&tk);
    tma_prefetch_map(&tv);
    sh.s_fail = 0;
  }
  // pairs with the wait before the cluster's first remote store: every peer runs by then
  if constexpr (CL) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait_then_release();

  // groups of 16 positions and units of a row
  auto groups_of = [&](int row) {
    if constexpr (!LIST) return (clamp_len(a.ctx_len[row / a.Hkv], a.Cap) + 15) >> 4;
    const int cnt = a.count ? a.count[row] : a.k_fixed;
    return min(max(cnt, 0), a.idx_stride) << (a.pshift - 4);
  };
  auto units_of = [&](int row) { return (groups_of(row) + SG - 1) / SG; };

  // the row holding unit x: the last row whose first unit (plus `beta` per
  // earlier row) is <= x
  auto row_at = [&](long long x, long long beta) {
    int l = 0, u = rows - 1;
    while (l < u) {
      const int mid = (l + u + 1) >> 1;
      if (s_pref[mid] + beta * mid <= x) l = mid;
      else u = mid - 1;
    }
    return l;
  };
  // First unit of CTA k's range: equal shares of a list in which each row start after the first counts
  // kPgSegCost tokens more, moved to the nearest start of a row if rows are not to be cut.  Short jobs use fewer CTAs.
  bool snap = false;
  auto range_start = [&](int k, int n) {
    const long long beta = kPgSegCost / UT, at = (s_pref[rows] + beta * (rows - 1)) * k / n;
    const int l = row_at(at, beta), first = s_pref[l], end = s_pref[l + 1], x = (int)min(at - beta * l, (long long)end);
    return !snap ? x : x - first <= end - x ? first : end;
  };
  // rows without units: output 0, lse -inf (or the sink alone)
  auto empty_rows = [&]() {
    for (int er = cta; er < rows; er += gridDim.x) {
      if (s_pref[er + 1] != s_pref[er]) continue;
      for (int i = threadIdx.x; i < G * D; i += NT)
        pg_finish<T, D>(a, (size_t)er * G + i / D, (er % a.Hkv) * G + i / D, kNegInf, 0.f, 0.f, i % D);
    }
  };

  int row = 0, lo = 0, hi = 0, grid = 1;
  if constexpr (CL) {
    row = cta / a.cluster;
    const int nu = units_of(row), split = cta % a.cluster;
    lo = (int)((long long)nu * split / a.cluster);
    hi = (int)((long long)nu * (split + 1) / a.cluster);
    __syncthreads();  // barriers initialised
  } else {
    // s_pref: exclusive prefix sum of the rows' units
    {
      const int rpt = (rows + NT - 1) / NT, r0 = threadIdx.x * rpt;
      int sum = 0, one = 0, longest = 0;  // one: the units of a thread's only row, read once
      for (int i = 0; i < rpt; ++i)
        if (r0 + i < rows) {
          sum += one = units_of(r0 + i);
          longest = max(longest, one);
        }
      longest = __reduce_max_sync(0xffffffffu, longest);
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) {
        sh.s_tmp[warp] = x;
        sh.s_tmp[16 + warp] = longest;
      }
      __syncthreads();
      int before = 0, total = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        before += w < warp ? sh.s_tmp[w] : 0;
        total += sh.s_tmp[w];
        longest = max(longest, sh.s_tmp[16 + w]);
      }
      constexpr int WHOLE = (int)(kPgWhole / (Tile::NS * UT));  // in units
      snap = longest <= 2 * WHOLE && longest - total / (int)gridDim.x <= WHOLE;
      int acc = before + x - sum;
      for (int i = 0; i < rpt; ++i)
        if (r0 + i < rows) {
          s_pref[r0 + i] = acc;
          acc += rpt == 1 ? one : units_of(r0 + i);
        }
      if (threadIdx.x == 0) s_pref[rows] = total;
      __syncthreads();
    }
    const int total = s_pref[rows];
    grid = min((int)gridDim.x, max(1, total / kPgMinUnits));
    if (cta < grid) {
      lo = range_start(cta, grid);
      hi = range_start(cta + 1, grid);
      row = row_at(lo, 0);
    }
    if (lo >= hi) {
      empty_rows();
      return;
    }
  }

  // the wait-timeout test hook: the first CTA with a unit (ranges of CTAs before it may be empty, and so may rows)
  bool plant = a.test_wait && lo == 0 && hi > 0 && warp == 0;
  if constexpr (CL)
    for (int r = 0; plant && r < row; ++r) plant = units_of(r) == 0;
  const uint32_t tries = plant ? kTestWaitTries : kWaitTries;
  const uint32_t wring = smem_u32(ring) + (uint32_t)warp * S * Tile::STAGE;
  uint32_t wseq = 0;  // this warp's ring position
  for (int e = lo; CL || e < hi;) {
    // segment ends in the CTA's own counting of units
    const int seg_end = CL ? hi : min(hi, s_pref[row + 1]), u0 = CL ? lo : e - s_pref[row];
    const int b = row / a.Hkv, h = row % a.Hkv;
    const int N = clamp_len(a.ctx_len[b], a.Cap), ng = groups_of(row);
    const int nseg = seg_end - e;
    const int nk = nseg > warp ? (nseg - warp + W - 1) / W : 0;  // this warp's units: u0 + warp + W k
    // a wait gave up: no more copies.  (One value for the warp: another warp may set it at any time.)
    const bool failed = __any_sync(0xffffffffu, sh.s_fail != 0);
    const int32_t* list = LIST ? a.page_idx + (size_t)row * a.idx_stride : nullptr;
    const int32_t* table = a.table + (size_t)b * MP;

    // Of unit kb + lane: where its groups' rows lie in the pool, and their valid tokens (0: nothing there).
    int at[SG], lim[SG];
    auto load_batch = [&](int kb) {
      const int k = kb + lane;
      unsigned bad = 0;
#pragma unroll
      for (int s = 0; s < SG; ++s) {
        at[s] = lim[s] = 0;
        const int g = (u0 + warp + W * k) * SG + s;
        if (k < nk && g < ng) {
          int pos = g << 4, lp = pos >> a.pshift;
          const int in = pos & (a.P - 1);
          // entries are counted once: by the unit holding the page's first group, when first loaded
          const bool once = in == 0 && (kb == 0 || lane >= S - 1);
          if constexpr (LIST) {
            lp = ld_global(list + lp);
            if ((unsigned)lp >= (unsigned)MP) {
              bad += once && lp != -1;
              continue;
            }
            pos = (lp << a.pshift) + in;
          }
          if (pos < N) {
            const int page = ld_global(table + lp);
            if (paged_page(page, a.pool)) {
              at[s] = ((page * a.Hkv + h) << a.pshift) + in;
              lim[s] = min(16, N - pos);
            } else {
              bad += once;
            }
          }
        }
      }
      note_bad_pages(bad);
    };
    // the copies of unit k (its batch entry in lane k - kb) into its stage
    auto issue = [&](int k, int kb) {
      int y[SG];
      bool there[SG];
      uint32_t bytes = 0;
#pragma unroll
      for (int s = 0; s < SG; ++s) {
        y[s] = __shfl_sync(0xffffffffu, at[s], k - kb);
        there[s] = __shfl_sync(0xffffffffu, lim[s], k - kb) > 0;
        if (there[s]) bytes += 2 * Tile::GROUP;
      }
      if (lane == 0) {
        const uint32_t st = (wseq + k) % S;
        uint64_t* bar = &full[warp][st];
        unsigned char* dst = ring + ((size_t)warp * S + st) * Tile::STAGE;
        if (plant && wseq + k == 0) {
          mbar_arrive_expect_tx(bar, 16);  // no copy is issued: this phase never completes
        } else if (bytes == 0) {
          mbar_arrive(bar);
        } else {
          mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
          for (int s = 0; s < SG; ++s)
            if (there[s]) {
              tma_load_3d(dst + s * Tile::GROUP, &tk, 0, y[s], 0, bar);
              tma_load_3d(dst + (SG + s) * Tile::GROUP, &tv, 0, y[s], 0, bar);
            }
        }
      }
    };

    bool ok = !failed;
    int k = 0;
    if (ok) {
      if (lane == 0) fence_proxy_async_smem();  // the merge's reads of the ring before the copies write it
      load_batch(0);
      for (int j = 0; j < min(S - 1, nk); ++j) issue(j, 0);
    }
    Tile tile;
    tile.start(static_cast<const T*>(a.q) + ((size_t)b * a.Hq + (size_t)h * G) * D, G, lane);
    if constexpr (!CL)
      if (e == lo) {  // while the first copies are on their way
        for (int c2 = threadIdx.x; c2 <= grid; c2 += NT) sh.s_lo[c2] = range_start(c2, grid);
        empty_rows();
      }
    for (int kb = 0; ok && kb < nk; kb += BATCH) {
      if (kb) load_batch(kb);
      const int kend = min(nk, kb + BATCH);
      for (; k < kend; ++k) {
        if (k + S - 1 < nk) issue(k + S - 1, kb);  // into the stage unit k - 1 has left
        const uint32_t st = (wseq + k) % S;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[warp][st], ((wseq + k) / S) & 1, tries))) {
          ok = false;
          break;
        }
        int n[SG], any = 0;
#pragma unroll
        for (int s = 0; s < SG; ++s) any |= n[s] = __shfl_sync(0xffffffffu, lim[s], k - kb);
        if (any) tile.unit(wring + st * Tile::STAGE, n, a.qscale, lane);
        // the stage is read before the copy engine may write it again
        __syncwarp();
        if (lane == 0) fence_proxy_async_smem();
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) {
      note_wait_timeout();
      sh.s_fail = 1;
      // the copies still in flight land before the ring is reused or left
      if (!failed)
        for (int k2 = k; k2 < min(nk, k + S); ++k2)
          mbar_wait(&full[warp][(wseq + k2) % S], ((wseq + k2) / S) & 1, tries);
    }
    wseq += failed ? 0u : (uint32_t)nk;
    __syncthreads();  // every warp's stages have been consumed (or drained): the rings become the merge area

    // a warp that gave up has an infinite maximum, which makes every later merge weight NaN
    float* sO = reinterpret_cast<float*>(ring);  // [W][8 heads][MROW]
    tile.finish(sO + warp * 8 * L::MROW, sM[warp], sL[warp], ok, lane);
    __syncthreads();
    if (threadIdx.x < 8) {
      const int g = threadIdx.x;
      float M = kNegInf, Lh = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, sM[w][g]);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        // a NaN sum without a maximum (every score NaN) is kept
        const float f = sM[w][g] == kNegInf ? (sL[w][g] == 0.f ? 0.f : 1.f) : pg_ex2(sM[w][g] - M);
        sF[w][g] = f;
        Lh = fmaf(sL[w][g], f, Lh);
      }
      if (Lh != Lh && M == kNegInf) M = 0.f;
      sHm[g] = M;
      sHl[g] = Lh;
    }
    __syncthreads();
    if constexpr (CL) {
      __shared__ PgInbox<D> inbox;
      namespace cg = cooperative_groups;
      cg::cluster_group cl = cg::this_cluster();
      const int C = a.cluster, split = cta % C, GD = G * D;
      const int chunk = ((GD + C - 1) / C + 3) & ~3;
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      for (int i = 4 * threadIdx.x; i < GD; i += 4 * NT) {
        const int g = i / D, d = i % D, owner = i / chunk;
        float4 av = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(sO + (w * 8 + g) * L::MROW + d);
          const float f = sF[w][g];
          av.x = fmaf(x.x, f, av.x);
          av.y = fmaf(x.y, f, av.y);
          av.z = fmaf(x.z, f, av.z);
          av.w = fmaf(x.w, f, av.w);
        }
        *reinterpret_cast<float4*>(cl.map_shared_rank(inbox.o, owner) + split * chunk + (i - owner * chunk)) = av;
      }
      if (threadIdx.x < C * G) {
        const int owner = threadIdx.x / G, g = threadIdx.x % G;
        cl.map_shared_rank(inbox.m, owner)[split * 8 + g] = sHm[g];
        cl.map_shared_rank(inbox.l, owner)[split * 8 + g] = sHl[g];
      }
      cl.sync();  // nothing remote is touched after this
      const int i1 = min(GD, (split + 1) * chunk);
      for (int i = split * chunk + threadIdx.x; i < i1; i += NT) {
        const int g = i / D;
        float M = kNegInf, Lh = 0.f, av = 0.f;
        for (int s = 0; s < C; ++s) M = fmaxf(M, inbox.m[s * 8 + g]);
        for (int s = 0; s < C; ++s) {
          const float ms = inbox.m[s * 8 + g];
          const float f = ms == kNegInf ? 0.f : pg_ex2(ms - M);
          Lh = fmaf(inbox.l[s * 8 + g], f, Lh);
          av = fmaf(inbox.o[s * chunk + (i - split * chunk)], f, av);
        }
        pg_finish<T, D>(a, (size_t)row * G + g, h * G + g, M, Lh, av, i % D);
      }
      return;
    }
    const bool whole = e == s_pref[row] && seg_end == s_pref[row + 1];
    const int slot = e == lo ? 2 * cta : 2 * cta + 1;
    for (int i = threadIdx.x; i < G * D; i += NT) {
      const int g = i / D, d = i % D;
      float av = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) av = fmaf(sO[(w * 8 + g) * L::MROW + d], sF[w][g], av);
      if (whole) {
        pg_finish<T, D>(a, (size_t)row * G + g, h * G + g, sHm[g], sHl[g], av, d);
      } else {
        const size_t sg = (size_t)slot * G + g;
        a.po[sg * D + d] = av;
        if (d == 0) {
          a.pm[sg] = sHm[g];
          a.pl[sg] = sHl[g];
        }
      }
    }
    if (!whole) {
      // the row's contributors are the CTAs from the one holding its first
      // unit to the one holding its last (those with units); CTA k wrote slot
      // 2k when its range starts inside the row, else 2k + 1
      __syncthreads();
      if (threadIdx.x == 0) {
        auto cta_of = [&](int x) {  // the last CTA whose range starts at or before unit x
          int l = 0, u = grid - 1;
          while (l < u) {
            const int mid = (l + u + 1) >> 1;
            if (sh.s_lo[mid] <= x) l = mid;
            else u = mid - 1;
          }
          return l;
        };
        const int cf = cta_of(s_pref[row]), cl = cta_of(s_pref[row + 1] - 1);
        int n = 0;
        for (int c2 = cf; c2 <= cl; ++c2)
          if (sh.s_lo[c2] < sh.s_lo[c2 + 1]) sh.s_slot[n++] = sh.s_lo[c2] >= s_pref[row] ? 2 * c2 : 2 * c2 + 1;
        sh.s_ncontrib = n;
        // one thread's fences cover the CTA's stores before the barrier and
        // its loads after the next one
        __threadfence();
        sh.s_last = atomicAdd(a.tickets + row, 1) == n - 1;
        __threadfence();
      }
      __syncthreads();
      if (sh.s_last) {
        const int n = sh.s_ncontrib;
        // a thread's first output: the first contributors' values are in flight while the weights are formed
        constexpr int U = 8;
        auto part = [&](int it, int jj) {
          return jj < n && it < G * (D / 4)
                     ? __ldcg(reinterpret_cast<const float4*>(a.po + ((size_t)sh.s_slot[jj] * G + it / (D / 4)) * D) + it % (D / 4))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = part(threadIdx.x, u);
        for (int g = warp; g < G; g += W) {
          constexpr int H = kPgWeights / 32;
          // the contributors' max and sum in registers, loaded at once
          float pm[H], pl[H];
#pragma unroll
          for (int u = 0; u < H; ++u) {
            const int jj = lane + 32 * u;
            pm[u] = jj < n ? __ldcg(a.pm + (size_t)sh.s_slot[jj] * G + g) : kNegInf;
            pl[u] = jj < n ? __ldcg(a.pl + (size_t)sh.s_slot[jj] * G + g) : 0.f;
          }
          float M = pm[0], Ls = 0.f;
#pragma unroll
          for (int u = 1; u < H; ++u) M = fmaxf(M, pm[u]);
          for (int jj = lane + kPgWeights; jj < n; jj += 32) M = fmaxf(M, __ldcg(a.pm + (size_t)sh.s_slot[jj] * G + g));
          M = warp_max(M);
          const float sk = a.sink ? a.sink[h * G + g] * kLog2e : kNegInf;
          M = fmaxf(M, sk);
          auto weight = [&](float ms) { return (ms == kNegInf || M == kNegInf) ? 0.f : pg_ex2(ms - M); };
#pragma unroll
          for (int u = 0; u < H; ++u) {
            const float w = weight(pm[u]);
            Ls += pl[u] * w;
            if (lane + 32 * u < n) sh.s_w[g][lane + 32 * u] = w;
          }
          for (int jj = lane + kPgWeights; jj < n; jj += 32) {
            const size_t sg = (size_t)sh.s_slot[jj] * G + g;
            Ls += __ldcg(a.pl + sg) * weight(__ldcg(a.pm + sg));
          }
          Ls = warp_sum(Ls);
          if (a.sink && M != kNegInf) Ls += pg_ex2(sk - M);
          if (lane == 0) {
            const float inv = Ls == 0.f ? 0.f : 1.f / Ls;  // NaN stays NaN
            const size_t hq = (size_t)row * G + g;
            sh.s_m[g] = M;
            sh.s_inv[g] = inv;
            if (a.lse) a.lse[hq] = Ls == 0.f ? kNegInf : M * kLn2 + logf(Ls);
          }
        }
        __syncthreads();
        for (int it = threadIdx.x; it < G * (D / 4); it += NT) {
          const int g4 = it / (D / 4), d4 = it % (D / 4);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int j0 = 0; j0 < n; j0 += U) {
            if (j0 || it >= NT)
#pragma unroll
              for (int u = 0; u < U; ++u) v[u] = part(it, j0 + u);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int jj = j0 + u;
              if (jj >= n) break;
              float w;
              if (jj < kPgWeights) {
                w = sh.s_w[g4][jj];
              } else {
                const float ms = __ldcg(a.pm + (size_t)sh.s_slot[jj] * G + g4);
                w = (ms == kNegInf || sh.s_m[g4] == kNegInf) ? 0.f : pg_ex2(ms - sh.s_m[g4]);
              }
              acc.x = fmaf(v[u].x, w, acc.x);
              acc.y = fmaf(v[u].y, w, acc.y);
              acc.z = fmaf(v[u].z, w, acc.z);
              acc.w = fmaf(v[u].w, w, acc.w);
            }
          }
          const float inv = sh.s_inv[g4];
          T* op = static_cast<T*>(a.out) + ((size_t)row * G + g4) * D + 4 * d4;
          op[0] = from_f32<T>(acc.x * inv);
          op[1] = from_f32<T>(acc.y * inv);
          op[2] = from_f32<T>(acc.z * inv);
          op[3] = from_f32<T>(acc.w * inv);
        }
        if (threadIdx.x == 0) a.tickets[row] = 0;  // ready for the next call
      }
    }
    __syncthreads();  // shared memory is reused by the next segment
    e = seg_end;
    ++row;
    while (row < rows && s_pref[row + 1] == s_pref[row]) ++row;  // empty rows hold no units
  }
}

// ------------------------------------------------------------------- launches

// The driver's tensor-map encoder, looked up once.
static PFN_cuTensorMapEncodeTiled_v12000 pg_encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return nullptr;
  }();
  return fn;
}

// The pool as [N * Hkv * P] rows in pieces of 128 bytes: a box is [piece][16 rows][128 bytes].
template <typename T, int D>
static bool pg_map(CUtensorMap* map, const void* base, uint64_t rows) {
  auto fn = pg_encode_fn();
  if (!fn) return false;
  constexpr int PC = 128 / sizeof(T), N = D / PC;
  cuuint64_t dims[3] = {PC, (cuuint64_t)rows, N};
  cuuint64_t strides[2] = {D * sizeof(T), 128};
  cuuint32_t box[3] = {PC, 16, N};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool paged_attend_supported(const Shape& s, const Paged& c) {
  return s.B * (long long)s.Hkv <= kPgMaxRows && (long long)s.B * s.Hkv * (s.Cap / 16 + 1) < (1ll << 30) &&
         (long long)c.pages * s.Hkv * s.P < (1ll << 31);
}

static int pg_grid() { return std::min(sm_count(), kPgMaxGrid); }
static size_t pg_256(size_t v) { return (v + 255) & ~(size_t)255; }

size_t paged_attend_workspace(const Shape& s) {
  const size_t slots = 2 * (size_t)pg_grid();
  return kPgTicketBytes + pg_256(slots * s.G * s.D * 4) + 2 * pg_256(slots * s.G * 4);
}

// What a launch of one kernel needs once per device: the limit of its dynamic
// shared memory raised, and the number of clusters of each size that fit.
struct PgDevice {
  std::atomic<int> clusters[kPgMaxCluster + 1];  // 0: not asked yet, else 1 + the number
  std::atomic<bool> raised;
};

template <typename Tile, bool LIST, bool CL>
static cudaError_t pg_prepare(PgDevice** out) {
  static PgDevice devices[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  PgDevice& d = devices[dev];
  if (!d.raised.load(std::memory_order_acquire)) {
    auto kern = paged_attend_kernel<Tile, LIST, CL>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)PgLayout<Tile>::smem(CL ? 0 : kPgMaxRows));
    if (e == cudaSuccess && CL) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    d.raised.store(true, std::memory_order_release);
  }
  *out = &d;
  return cudaSuccess;
}

// Clusters of c CTAs of the cluster kernel that run at once (asked once per device).
template <typename Tile, bool LIST>
static int pg_clusters(int c, PgDevice* d) {
  int n = d->clusters[c].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(Tile::W * 32);
    cfg.dynamicSmemBytes = PgLayout<Tile>::smem(0);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int got = 0;
    if (cudaOccupancyMaxActiveClusters(&got, paged_attend_kernel<Tile, LIST, true>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      got = 0;
    }
    n = 1 + got;
    d->clusters[c].store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

// CTAs per row of the cluster kernel, or 0 for ranges over all rows, by their costs.  A
// CTA takes Tile::NS ns a token and a cluster 5.3 us besides, in as many waves as the clusters need; the
// ranges take 12 us, 3 per row of a CTA, and 23 / rows for rows that many CTAs share; both read at the
// memory's rate at most (near it a cluster's two bounds add up as their cubes' root).
// `most` bounds a row's tokens; where only the device knows them, rows are taken to hold four fifths
// of it on average and a cluster to wait for one that is full.  Measured on 260 shapes of 1 to 256
// rows, full and with lengths spread evenly from none: 16.9 us with two CTAs a row and 20 in ranges
// for 64 lists of 2048 tokens, 25.7 and 32.1 for 64 full rows of 4k, 188 and 167 for 64 uneven ones of
// up to 64k.  Nine in ten shapes take within 8% of the faster side, the others lose up to a quarter (64 full fp32
// rows of 4k at D = 128: 61 us, 50 with two CTAs a row).
template <typename Tile, bool LIST>
static int pg_pick(int rows, double most, bool fixed, bool even, PgDevice* d) {
  const double t = Tile::NS * 1e-3, sms = sm_count();
  const double mean = fixed ? most : 0.8 * most, longest = even ? mean : most;
  const double memory = rows * 2.0 * Tile::D * sizeof(typename Tile::T) / 6.7e6;  // us a token of every row
  double best = 12.0 + 3.0 * rows / sms + mean * std::max(memory, rows / sms * t) + 23.0 / rows;
  int pick = 0;
  for (int c = 1; c <= kPgMaxCluster; ++c) {
    const int n = c == 1 ? sm_count() : pg_clusters<Tile, LIST>(c, d);
    if (n < 1) continue;
    const int waves = (rows + n - 1) / n;
    const double us = waves * 5.3 + std::cbrt(std::pow(waves * longest * t / c, 3.0) + std::pow(mean * memory, 3.0));
    if (us < best) {
      best = us;
      pick = c;
    }
  }
  return pick;
}

template <typename Tile, bool LIST>
static cudaError_t pg_launch(PagedAttend a, const Paged& c, cudaStream_t st) {
  using L = PgLayout<Tile>;
  CUtensorMap tk, tv;
  const uint64_t rows = (uint64_t)c.pages * a.Hkv * a.P;
  if (!pg_map<typename Tile::T, Tile::D>(&tk, c.k, rows) || !pg_map<typename Tile::T, Tile::D>(&tv, c.v, rows))
    return cudaErrorInvalidValue;
  PgDevice* d;
  cudaError_t e = pg_prepare<Tile, LIST, true>(&d);
  if (e != cudaSuccess) return e;
  const bool fixed = LIST && !a.count;  // lists of one length; one sequence's rows are of one length too
  const double most = LIST ? (double)(a.count ? a.idx_stride : a.k_fixed) * a.P : a.Cap;
  a.cluster = pg_pick<Tile, LIST>(a.rows, most, fixed, fixed || (!LIST && a.rows == a.Hkv), d);
  if (a.cluster)
    return launch_pdl_cluster(paged_attend_kernel<Tile, LIST, true>, dim3(a.rows * a.cluster), dim3(Tile::W * 32), L::smem(0),
                              a.cluster, st, tk, tv, a);
  if ((e = pg_prepare<Tile, LIST, false>(&d)) != cudaSuccess) return e;
  return launch_pdl(paged_attend_kernel<Tile, LIST, false>, dim3(pg_grid()), dim3(Tile::W * 32), L::smem(a.rows), st, tk, tv, a);
}

template <bool LIST>
static cudaError_t pg_dispatch(const Shape& s, const PagedAttend& a, const Paged& c, cudaStream_t st) {
  if (s.dtype == 0) {
    if (s.G <= 4) return s.D == 64 ? pg_launch<PgF32<64, 4>, LIST>(a, c, st) : pg_launch<PgF32<128, 4>, LIST>(a, c, st);
    return s.D == 64 ? pg_launch<PgF32<64, 8>, LIST>(a, c, st) : pg_launch<PgF32<128, 8>, LIST>(a, c, st);
  }
  return s.D == 64 ? pg_launch<PgBf16<64>, LIST>(a, c, st) : pg_launch<PgBf16<128>, LIST>(a, c, st);
}

cudaError_t launch_paged_attend(const Shape& s, const Paged& c, const void* q, const int32_t* page_idx, int idx_stride,
                                const int32_t* count, int k_fixed, const float* sink, void* out, float* lse, void* ws,
                                cudaStream_t st) {
  PagedAttend a = {};
  a.q = q;
  a.table = c.table;
  a.page_idx = page_idx;
  a.count = count;
  a.ctx_len = c.ctx;
  a.idx_stride = idx_stride;
  a.k_fixed = k_fixed;
  a.rows = s.B * s.Hkv;
  a.Hq = s.Hq; a.Hkv = s.Hkv; a.G = s.G; a.Cap = s.Cap; a.P = s.P; a.pshift = s.pshift; a.pool = c.pages;
  a.test_wait = (s.flags & kFlagTestWaitTimeout) ? 1 : 0;
  a.qscale = s.scale * kLog2e;
  a.sink = sink;
  a.out = out;
  a.lse = lse;
  const size_t slots = 2 * (size_t)pg_grid();
  char* w = static_cast<char*>(ws);
  a.tickets = reinterpret_cast<int32_t*>(w);
  w += kPgTicketBytes;
  a.po = reinterpret_cast<float*>(w);
  w += pg_256(slots * s.G * s.D * 4);
  a.pm = reinterpret_cast<float*>(w);
  w += pg_256(slots * s.G * 4);
  a.pl = reinterpret_cast<float*>(w);
  const cudaError_t e = page_idx ? pg_dispatch<true>(s, a, c, st) : pg_dispatch<false>(s, a, c, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

DeviceStatus take_status_attend_paged() { return take_status_here(); }

}  // namespace sls
