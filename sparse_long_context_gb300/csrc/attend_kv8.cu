// Decode attention over the 8-bit cache (codes times a scale per block of
// tokens and head; the newest, partial block in bf16 in its tail buffer).
//
// The G query heads of a KV head share every byte read.  A row's tokens are
// taken in units of 16 SG positions (whole pages of a list, or the context in
// order); the rows' units, concatenated, are cut into one nearly equal range
// per CTA (one CTA per SM), so that rows of uneven length fill the GPU, and the
// last CTA to finish a shared row merges its partials in CTA order.
//
// A unit is streamed by one warp through its own ring of shared-memory stages
// (K codes, then V codes, one tensor-map box of 16 SG rows each, or SG boxes
// where pages have 16 tokens), so a late copy holds up one warp only.  Both
// products run on the fp16 tensor cores with the codes as exact operands:
//   S^T = Q K^T    A = the heads' queries, scaled to at most 2^11 by a power of
//                  two of their own (exact but for parts below 2^-35 of the
//                  head's largest, which round to fp16's subnormals), B = codes
//   x   = S * scale * s_k          fp32, one multiplication per score
//   O^T += V^T W^T,  W = p s_v     rounded to fp16 (half a step, 2^-11: independent
//                  errors of a row's weights, which add 2.6e-4 of the output to the 1.7e-3
//                  of its own rounding to bf16; a second part would double the products)
// The running maximum is that of x + e - 14 with 2^e <= s_v < 2^(e+1) the exponent of
// the value scale: then W = exp2(x - m) s_v < 2^15 for blocks of any scale, nothing
// overflows, and the largest W is 2^14 or more, so that weights down to 2^-28 of it
// keep their bits and what underflows is below 2^-38 of it.  (e is held within
// [-80, 121], so that exp2(x - m) and its sum over 2^31 tokens stay finite as well;
// scales below 2^-108 lose bits, those below 2^-119 add nothing.)  Sum and maximum are
// consistent, so the merge and the sink need no other form.  Tail tokens go through the
// bf16 tensor cores (weights in a high and a low part, half a step 2^-15), a group of
// 16 with the exponent of the scale that its values would be stored with.
//
// Bound by memory on long contexts: 32 contexts of 49k to 64k tokens, 2 KV heads of 6
// query heads and 128 channels, int8: 140 to 143 us for 943 MB (6.6 to 6.7 TB/s, the
// measured copy rate); e4m3 is 6% slower, its conversion instruction the busiest
// pipe.  At D = 64 the work per token weighs twice as much: 81 us for 470 MB (85%).
// Short rows are bound by a chain of latencies (lengths, list, scales, copies, merge):
// 6.2 us for 1000 tokens of 4 heads, 12 us for 128 pages of 16 tokens in 64 rows.
// Rows of middle length stay far from the copy rate: 26 us for 4 rows of 64k tokens (a
// cluster of 16 CTAs each, floor 10), and the variant follows from the capacity, so 64
// rows of 1000 tokens take 8 us in a capacity of 1024 and 14 in 65536.  (Times of the
// device alone, calls replayed from a graph.)
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "attend_common.cuh"
#include "kv8.cuh"
#include "launch.h"
#include "mma.cuh"
#include "tma.cuh"

namespace sls {

constexpr int kKv8MaxGrid = 1024;  // CTAs whose ranges are kept in shared memory
constexpr int kKv8MaxCluster = 16;
constexpr int kKv8MaxRows = 4096;  // rows whose first units are kept there
// The arrival counters' place in a workspace, whatever the shape: no call's partials lie
// where another one's counters are.
constexpr size_t kKv8TicketBytes = kKv8MaxRows * sizeof(int32_t);
constexpr int kKv8PerSm = 1;       // resident CTAs of an SM
// Least units of a CTA in ranges: a shorter job uses fewer CTAs.  2, 4 and 8 units: 10.8,
// 11.5 and 13.1 us for 8 rows of 1000 tokens in a capacity of 131072, 10.8, 10.6 and 15.8
// for 32 rows of 500 at D = 64; 64 rows of 100 tokens would be faster with 2 (7.4, 11.7
// and 20.5), rows of 4000 take the same with each.
constexpr int kKv8MinUnits = 4;
// Work of a row change (drain, merge, partial and refill) in tokens: 512 to 4096
// measured on seven shapes, 2048 the best or within 2% of it on six (64k x 32 dense
// 142 us at 1024, 140 at 2048, 144 at 4096).
constexpr int kKv8SegCost = 2048;

struct Kv8Attend {
  Kv8 c;
  const bf16* q;
  const int32_t *page_idx, *count, *ctx_len;
  int idx_stride, k_fixed, rows, Hq, Hkv, G, Cap, P, pshift, boxes, test_wait, cluster;
  float qscale;  // softmax scale * log2(e)
  const float* sink;
  bf16* out;
  float* lse;
  int32_t* tickets;     // [rows] arrival counters, zero between calls
  float *po, *pm, *pl;  // [slot][G][D], [slot][G] partials, two slots per CTA, max in base-2 units
  float2* grp;          // [rows, G, Cap >> gshift] weight sums of 2^gshift tokens and the max they are relative to
  int gshift;           // a unit's tokens, or a block's where blocks are smaller
  float2* fin;          // [B, Hq] final max (base 2) and 1 / sum
  const float* mass_in;
  float* mass_out;
};

__device__ __forceinline__ float kv8_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void kv8_mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t kv8_h2(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Four codes as two fp16x2 of their exact values.  int8: the code plus 128 in
// the low byte under the exponent 0x64 reads as 1152 + code.
template <int FMT>
__device__ __forceinline__ void kv8_unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kKv8Int8) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 k = __float2half2_rn(1152.f);
    uint32_t x = __byte_perm(u, 0x64646464u, 0x4140u), y = __byte_perm(u, 0x64646464u, 0x4342u);
    lo = kv8_h2(__hsub2(*reinterpret_cast<__half2*>(&x), k));
    hi = kv8_h2(__hsub2(*reinterpret_cast<__half2*>(&y), k));
  } else {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// What a value scale adds to its scores in the running maximum: its exponent, within
// [-80, 121] (0 gives -80; NaN and inf 121), less 14, so that the largest weight takes
// fp16's upper range and those far below it stay clear of its subnormals.
__device__ __forceinline__ float kv8_exponent(float s) {
  const int e = (int)((__float_as_uint(s) >> 23) & 255u) - 127;
  return (float)(min(max(e, -80), 121) - 14);
}

template <int D, int SG, int W, int S>
struct Kv8Layout {
  static constexpr int GROUP = 16 * D;                    // bytes of a group's K (or V) codes
  static constexpr int STAGE = 2 * SG * GROUP;            // K of the unit's groups, then V
  static constexpr size_t RING = (size_t)W * S * STAGE;
  // The warps' accumulators, [warp][head][D + 4]: the lanes of a warp then
  // write to different banks (kv8_channel gives the order of the channels).
  static constexpr int MROW = D + 4;
  static constexpr size_t MERGE = (size_t)W * 8 * MROW * sizeof(float);
  static constexpr size_t REGION = RING > MERGE ? RING : MERGE;
};

// Shared-memory offset of 16-byte chunk c of row t of a box (the copy
// engine's 128-byte swizzle for 128-byte rows, 64-byte swizzle for 64-byte rows:
// eight consecutive rows' same chunk lies in eight different bank groups).
template <int D>
__device__ __forceinline__ int kv8_chunk(int t, int c) {
  return D == 128 ? t * 128 + ((c ^ (t & 7)) << 4) : t * 64 + ((c ^ ((t >> 1) & 3)) << 4);
}

// Channel held at place p of an accumulator row in shared memory and in the
// partials: m-tile t's rows r and r + 8 are channels r D/8 + 2t and + 1, at
// places 16 t + 2 r and + 1.
template <int D>
__device__ __forceinline__ int kv8_channel(int p) {
  return ((p & 15) >> 1) * (D / 8) + 2 * (p >> 4) + (p & 1);
}

// Scores of one stored group: lane (r, m) gets head r, tokens 2m, 2m+1 (sc[0])
// and 8+2m, 9+2m (sc[1]).  The k slots of step c hold channels 16c + 4m .. + 3
// of lane m (the order of a sum is free), so one ldmatrix register is the four
// codes of both B registers.
template <int D, int FMT>
__device__ __forceinline__ void kv8_scores(uint32_t k, const uint32_t (&qa)[D / 16][2], float (&sc)[2][4], int lane) {
  const int j = lane >> 3, tok = 8 * (j & 1) + (lane & 7);
#pragma unroll
  for (int i = 0; i < 4; ++i) sc[0][i] = sc[1][i] = 0.f;
#pragma unroll
  for (int c = 0; c < D / 16; c += 2) {
    uint32_t w[4];
    ldsm_x4(k + kv8_chunk<D>(tok, c + (j >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b0, b1;
      kv8_unpack4<FMT>(w[i], b0, b1);
      kv8_mma_f16(sc[i & 1], qa[c + (i >> 1)][0], 0u, qa[c + (i >> 1)][1], 0u, b0, b1);
    }
  }
}

// O^T += V^T W^T of one stored group.  Lane (r, m) reads channels
// [r D/8, (r+1) D/8) of tokens 2m, 2m+1, 8+2m, 9+2m; m-tile t takes its channels
// 2t (row r) and 2t + 1 (row r + 8).
template <int D, int FMT>
__device__ __forceinline__ void kv8_pv(uint32_t v, float (&o)[D / 16][4], uint32_t p0, uint32_t p1, int lane) {
  constexpr int NW = D / 32;  // 32-bit words of a lane's channels
  const int r = lane >> 2, m = lane & 3;
  uint32_t w[4][NW];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 2 * m + (i & 1) + 8 * (i >> 1);
    if constexpr (D == 128) {
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                   : "r"(v + kv8_chunk<D>(t, r)));
    } else {
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                   : "=r"(w[i][0]), "=r"(w[i][1])
                   : "r"(v + kv8_chunk<D>(t, r >> 1) + 8 * (r & 1)));
    }
  }
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    uint32_t a[2][4];  // [token pair][byte]: the two tokens' values of one channel
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      kv8_unpack4<FMT>(__byte_perm(w[2 * u][k], w[2 * u + 1][k], 0x5140u), a[u][0], a[u][1]);
      kv8_unpack4<FMT>(__byte_perm(w[2 * u][k], w[2 * u + 1][k], 0x7362u), a[u][2], a[u][3]);
    }
    kv8_mma_f16(o[2 * k], a[0][0], a[0][1], a[1][0], a[1][1], p0, p1);
    kv8_mma_f16(o[2 * k + 1], a[0][2], a[0][3], a[1][2], a[1][3], p0, p1);
  }
}

// A group of the tail buffer (bf16, `lim` valid tokens; the others are not
// read and count as zero).  All of its loads are issued together: a CTA meets
// it once per row, with the memory system busy.
template <int D>
struct Kv8Tail {
  uint2 k[2][D / 16];
  uint32_t v[4][D / 16];
  int lim;
  __device__ __forceinline__ void load(const bf16* kt, const bf16* vt, int n, int lane) {
    const int r = lane >> 2, m = lane & 3;
    lim = n;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int t = r + 8 * nt;
        k[nt][c] = t < lim ? *reinterpret_cast<const uint2*>(kt + (size_t)t * D + 16 * c + 4 * m) : make_uint2(0u, 0u);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 2 * m + (i & 1) + 8 * (i >> 1);
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {  // the lane's D/8 channels in 16-byte loads
        const uint4 x = t < lim ? *reinterpret_cast<const uint4*>(vt + (size_t)t * D + r * (D / 8) + 8 * u)
                                : make_uint4(0u, 0u, 0u, 0u);
        v[i][4 * u] = x.x; v[i][4 * u + 1] = x.y; v[i][4 * u + 2] = x.z; v[i][4 * u + 3] = x.w;
      }
    }
  }
  // The exponent with which the group's values enter the running maximum: that of
  // the scale they would be stored with, so that a token weighs the same in the
  // tail and in a block.  Infinities and NaN are left out: they show in their own
  // channels and must not push the others' weights down.
  template <int FMT>
  __device__ __forceinline__ float exponent() const {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint32_t a = v[i][c] & 0x7fff7fffu;
        mx = __vmaxu2(mx, a & __vcmpltu2(a, 0x7f807f80u));
      }
    mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    return kv8_exponent(__uint_as_float(mx << 16) * (1.f / kv8_top<FMT>()));
  }
  // q: channels 16 c + 4 m .. + 3 of the lane's head
  __device__ __forceinline__ void scores(const uint2 (&q)[D / 16], float mul, float (&x)[4], int lane) const {
    const int m = lane & 3;
    float sc[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[0][i] = sc[1][i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) mma_bf16(sc[nt], q[c].x, 0u, q[c].y, 0u, k[nt][c].x, k[nt][c].y);
    x[0] = 2 * m < lim ? sc[0][0] * mul : kNegInf;
    x[1] = 2 * m + 1 < lim ? sc[0][1] * mul : kNegInf;
    x[2] = 2 * m + 8 < lim ? sc[1][0] * mul : kNegInf;
    x[3] = 2 * m + 9 < lim ? sc[1][1] * mul : kNegInf;
  }
  // O^T += V^T P^T with the weights as the sum of two bf16 (16 bits in all, half a step
  // 2^-15: the tail may be a whole context, and the newest tokens draw much weight).  The
  // high part is truncated, so the low one has its sign, and a low part of zero becomes
  // 2^-126 next to a weight, so that no infinite value meets a zero or another sign.
  __device__ __forceinline__ void pv(float (&o)[D / 16][4], const float (&p)[4]) const {
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      hi[i] = __byte_perm(__float_as_uint(p[2 * i]), __float_as_uint(p[2 * i + 1]), 0x7632);
      lo[i] = pack_bf16(p[2 * i] - bf16lo(hi[i]), p[2 * i + 1] - bf16hi(hi[i]));
      lo[i] = __vmaxu2(lo[i], 0x00800080u) & __vcmpgtu2(hi[i], 0u);
    }
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const uint32_t a0 = __byte_perm(v[0][t], v[1][t], 0x5410), a1 = __byte_perm(v[0][t], v[1][t], 0x7632);
      const uint32_t a2 = __byte_perm(v[2][t], v[3][t], 0x5410), a3 = __byte_perm(v[2][t], v[3][t], 0x7632);
      mma_bf16(o[t], a0, a1, a2, a3, hi[0], hi[1]);
      mma_bf16(o[t], a0, a1, a2, a3, lo[0], lo[1]);
    }
  }
};

constexpr int kKv8Weights = 160;  // contributors of a row whose weights are kept (all SMs of a GB300)
template <bool CL>
struct Kv8Smem {
  int s_lo[CL ? 1 : kKv8MaxGrid + 1];  // first unit of every CTA's range, and the total
  int s_slot[CL ? 1 : kKv8MaxGrid];
  int s_tmp[32];
  int s_fail, s_ncontrib, s_last;
  float s_w[8][CL ? 1 : kKv8Weights], s_m[8], s_inv[8];
};

// Final output of head g, channel d: accumulator av and sum lv relative to
// exp2(M); the sink joins the sum.
template <int D>
__device__ __forceinline__ void kv8_finish(const Kv8Attend& a, size_t hq, int head, float M, float lv, float av, int d) {
  const float sk = a.sink ? a.sink[head] * kLog2e : kNegInf;
  const float Mx = fmaxf(M, sk);
  float f = 0.f, Lt = 0.f;
  if (Mx != kNegInf) {
    f = M == kNegInf ? 0.f : kv8_ex2(M - Mx);
    Lt = lv * f + (a.sink ? kv8_ex2(sk - Mx) : 0.f);
  }
  // a NaN sum (a NaN block, or a wait that gave up) stays NaN in the output and lse
  a.out[hq * D + d] = __float2bfloat16_rn(Lt == 0.f ? 0.f : __fdividef(av * f, Lt));  // Lt < 2^126: two ulp
  if (d == 0) {
    if (a.lse) a.lse[hq] = Lt == 0.f ? kNegInf : Mx * kLn2 + logf(Lt);
    if (a.fin) a.fin[hq] = make_float2(Mx, Lt == 0.f ? 0.f : 1.f / Lt);
  }
}

// What the CTAs of a row's cluster send each other: rank r merges its share of
// the G x D outputs, a multiple of 4 values.
template <int D>
struct __align__(16) Kv8Inbox {
  float o[8 * D + 4 * kKv8MaxCluster];
  float m[kKv8MaxCluster * 8], l[kKv8MaxCluster * 8];
};

// CL: the CTAs of a cluster take one row's units in equal shares and merge
// through distributed shared memory; otherwise every CTA takes a range of all
// rows' units.
template <int D, int FMT, int SG, int W, int S, bool LIST, bool MASS, bool CL>
__global__ void __launch_bounds__(W * 32, kKv8PerSm)
kv8_attend_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Kv8Attend a) {
  using L = Kv8Layout<D, SG, W, S>;
  constexpr int KS = D / 16, NT = W * 32, UT = 16 * SG;
  constexpr int BATCH = 32 - (S - 1);  // units between two loads of a warp's page ids and scales
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  int* s_pref = reinterpret_cast<int*>(ring + L::REGION);  // [rows + 1] first unit of each row
  __shared__ Kv8Smem<CL> sh;
  __shared__ uint64_t full[W][S];
  __shared__ float sM[W][8], sL[W][8], sF[W][8], sHm[8], sHl[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, m = lane & 3;
  const int G = a.G, rows = a.rows, cta = blockIdx.x;
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

  // Groups and units of a row.  Dense: the groups of its complete blocks; the
  // tail's go with the last unit (a row with nothing but a tail has one unit).
  auto groups_of = [&](int row) {
    if constexpr (!LIST)
      return clamp_len(a.ctx_len[row / a.Hkv], a.Cap) >> a.c.bshift << (a.c.bshift - 4);
    const int cnt = a.count ? a.count[row] : a.k_fixed;
    return min(max(cnt, 0), a.idx_stride) << (a.pshift - 4);
  };
  auto units_of = [&](int row) {
    const int n = (groups_of(row) + SG - 1) / SG;
    return LIST || n > 0 ? n : (a.ctx_len[row / a.Hkv] > 0 ? 1 : 0);
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
    int sum = 0, one = 0;  // one: the units of a thread's only row, read once
    for (int i = 0; i < rpt; ++i)
      if (r0 + i < rows) sum += one = units_of(r0 + i);
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh.s_tmp[warp] = x;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      before += w < warp ? sh.s_tmp[w] : 0;
      total += sh.s_tmp[w];
    }
    int acc = before + x - sum;
    for (int i = 0; i < rpt; ++i)
      if (r0 + i < rows) {
        s_pref[r0 + i] = acc;
        acc += rpt == 1 ? one : units_of(r0 + i);
      }
    if (threadIdx.x == 0) s_pref[rows] = total;
    __syncthreads();
  }
  const int T = s_pref[rows];
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
  // Every CTA's range: equal shares of a list in which each row start after
  // the first counts kKv8SegCost tokens more.  Short jobs use fewer CTAs.
  grid = min((int)gridDim.x, max(1, T / kKv8MinUnits));
  {
    const long long beta = kKv8SegCost / UT, Tp = T + beta * (rows - 1);
    for (int k = threadIdx.x; k <= grid; k += NT) {
      const long long at = Tp * k / grid;
      const int l = row_at(at, beta);
      sh.s_lo[k] = (int)min(at - beta * l, (long long)s_pref[l + 1]);
    }
  }
  __syncthreads();
  // rows without units: output 0, lse -inf (or the sink alone)
  for (int er = cta; er < rows; er += gridDim.x) {
    if (s_pref[er + 1] != s_pref[er]) continue;
    for (int i = threadIdx.x; i < G * D; i += NT)
      kv8_finish<D>(a, (size_t)er * G + i / D, (er % a.Hkv) * G + i / D, kNegInf, 0.f, 0.f, i % D);
  }
  if (cta >= grid) return;
  lo = sh.s_lo[cta];
  hi = sh.s_lo[cta + 1];
  if (lo >= hi) return;
  row = row_at(lo, 0);
  }

  const bool plant = a.test_wait && cta == 0 && warp == 0;  // the wait-timeout test hook
  const uint32_t tries = plant ? kTestWaitTries : kWaitTries;
  const uint32_t wring = smem_u32(ring) + (uint32_t)warp * S * L::STAGE;
  uint32_t wseq = 0;  // this warp's ring position
  for (int e = lo; CL || e < hi;) {
    // segment ends and row ends in the CTA's own counting of units
    const int row_end = CL ? units_of(row) : s_pref[row + 1];
    const int seg_end = CL ? hi : min(hi, row_end), u0 = CL ? lo : e - s_pref[row];
    const int b = row / a.Hkv, h = row % a.Hkv;
    const int N = clamp_len(a.ctx_len[b], a.Cap), ng = groups_of(row), newest = N >> a.c.bshift;
    const int nseg = seg_end - e;
    const int nk = nseg > warp ? (nseg - warp + W - 1) / W : 0;  // this warp's units: u0 + warp + W k
    const bool failed = sh.s_fail != 0;                          // an earlier segment gave up: no more copies
    const int32_t* list = LIST ? a.page_idx + (size_t)row * a.idx_stride : nullptr;
    const size_t row_blk = (size_t)row * (a.Cap >> a.c.bshift);

    const bf16* qh = a.q + ((size_t)b * a.Hq + (size_t)h * G + r) * D;
    // the lane's part of its head's query
    auto load_q = [&](uint2 (&raw)[KS]) {
#pragma unroll
      for (int c = 0; c < KS; ++c)
        raw[c] = r < G ? __ldg(reinterpret_cast<const uint2*>(qh + 16 * c + 4 * m)) : make_uint2(0u, 0u);
    };
    uint32_t qa[KS][2];
    float qmul;
    float o[KS][4], m_run = kNegInf, l_run = 0.f;
#pragma unroll
    for (int t = 0; t < KS; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    // Takes the lane's new maximum into the running one and rescales sum and
    // accumulators; returns the value the weights are relative to.
    auto softmax_step = [&](float gm) {
      gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));
      gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
      const float mn = fmaxf(m_run, gm), mref = mn == kNegInf ? 0.f : mn;
      const float alpha = kv8_ex2(m_run - mref);  // before any token: exp2(-inf) = 0 scales zeros
      m_run = mn;
      l_run *= alpha;
      // accumulator columns are heads 2m and 2m + 1
      const float a_lo = __shfl_sync(0xffffffffu, alpha, 8 * m), a_hi = __shfl_sync(0xffffffffu, alpha, 8 * m + 4);
      if (!__all_sync(0xffffffffu, a_lo == 1.f && a_hi == 1.f)) {
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          o[t][0] *= a_lo; o[t][1] *= a_hi; o[t][2] *= a_lo; o[t][3] *= a_hi;
        }
      }
      return mref;
    };
    // the 16 positions from `at` on, which lie in the tail buffer
    auto tail_group = [&](int at) {
      uint2 q[KS];
      load_q(q);
      const size_t tail = ((size_t)row * a.c.block + (at & (a.c.block - 1))) * D;
      Kv8Tail<D> g;
      g.load(static_cast<const bf16*>(a.c.kt) + tail, static_cast<const bf16*>(a.c.vt) + tail, min(16, N - at), lane);
      float x[4];
      g.scores(q, a.qscale, x, lane);
      const float mref = softmax_step(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) + g.template exponent<FMT>());
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = kv8_ex2(x[i] - mref);
      l_run += (x[0] + x[1]) + (x[2] + x[3]);
      g.pv(o, x);
    };

    // Of unit kb + lane: the positions of its groups (-1: nothing there) and
    // the scales of those in complete blocks.
    int base[SG];
    float ksc[SG], vsc[SG];
    auto load_batch = [&](int kb) {
      const int k = kb + lane;
      unsigned bad = 0;
#pragma unroll
      for (int s = 0; s < SG; ++s) {
        base[s] = -1;
        ksc[s] = vsc[s] = 1.f;
        const int g = (u0 + warp + W * k) * SG + s;
        if (k < nk && g < ng) {
          int at = g << 4;
          if constexpr (LIST) {
            const int pg = __ldg(list + (at >> a.pshift)), in = at & (a.P - 1);
            // counted once: by the unit holding the page's first group, when first loaded
            bad += in == 0 && (kb == 0 || lane >= S - 1) && bad_page_id(pg, a.Cap >> a.pshift);
            at = (unsigned)pg < (unsigned)(a.Cap >> a.pshift) ? (pg << a.pshift) + in : a.Cap;
          }
          if (at < N) {
            base[s] = at;
            if (at >> a.c.bshift < newest) {
              ksc[s] = __ldg(a.c.ks + row_blk + (at >> a.c.bshift));
              vsc[s] = __ldg(a.c.vs + row_blk + (at >> a.c.bshift));
            }
          }
        }
      }
      if constexpr (LIST) note_bad_pages(bad);
    };
    // the copies of unit k (its batch entry in lane k - kb) into its stage
    auto issue = [&](int k, int kb) {
      int at[SG];
      uint32_t bytes = 0;
#pragma unroll
      for (int s = 0; s < SG; ++s) {
        at[s] = __shfl_sync(0xffffffffu, base[s], k - kb);
        if (at[s] >= 0 && at[s] >> a.c.bshift >= newest) at[s] = -1;  // tail tokens are not copied
        if (at[s] >= 0) bytes += 2 * L::GROUP;
      }
      if (lane == 0) {
        const uint32_t st = (wseq + k) % S;
        uint64_t* bar = &full[warp][st];
        unsigned char* dst = ring + ((size_t)warp * S + st) * L::STAGE;
        if (plant && wseq + k == 0) {
          mbar_arrive_expect_tx(bar, 16);  // no copy is issued: this phase never completes
        } else if (bytes == 0) {
          mbar_arrive(bar);
        } else if (a.boxes == 1) {  // one box of the unit's 16 SG rows (at[0] >= 0 when any is)
          mbar_arrive_expect_tx(bar, L::STAGE);
          tma_load_2d(dst, &tk, 0, row * a.Cap + at[0], bar);
          tma_load_2d(dst + SG * L::GROUP, &tv, 0, row * a.Cap + at[0], bar);
        } else {
          mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
          for (int s = 0; s < SG; ++s)
            if (at[s] >= 0) {
              tma_load_2d(dst + s * L::GROUP, &tk, 0, row * a.Cap + at[s], bar);
              tma_load_2d(dst + (SG + s) * L::GROUP, &tv, 0, row * a.Cap + at[s], bar);
            }
        }
      }
    };

    bool ok = !failed;
    int k = 0;
    uint2 raw[KS];
    if constexpr (LIST) load_q(raw);  // in flight with the list (the dense kernels start their copies first)
    if (ok) {
      if (lane == 0) fence_proxy_async_smem();  // the merge's reads of the ring before the copies write it
      load_batch(0);
      for (int j = 0; j < min(S - 1, nk); ++j) issue(j, 0);
      if constexpr (!LIST) {
        // the row's last CTA: its tail groups, one per warp from the last warp down
        if (seg_end == row_end)
          for (int at = (newest << a.c.bshift) + 16 * (W - 1 - warp); at < N; at += 16 * W) tail_group(at);
      }
    }
    if constexpr (!LIST) load_q(raw);
    // the heads' queries as fp16 with their largest channel in [2^10, 2^11)
    {
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < KS; ++c) mx = __vmaxu2(mx, __vmaxu2(raw[c].x & 0x7fff7fffu, raw[c].y & 0x7fff7fffu));
      mx = max(mx & 0xffffu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int ex = (int)(mx >> 7) - 127;  // 128 for infinity and NaN, -127 for zero and subnormals
      const int sh2 = ex == 128 ? 0 : min(10 - ex, 100);
      const float f = __uint_as_float((uint32_t)(sh2 + 127) << 23);
      qmul = a.qscale * __uint_as_float((uint32_t)(127 - sh2) << 23);
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        qa[c][0] = kv8_h2(__floats2half2_rn(bf16lo(raw[c].x) * f, bf16hi(raw[c].x) * f));
        qa[c][1] = kv8_h2(__floats2half2_rn(bf16lo(raw[c].y) * f, bf16hi(raw[c].y) * f));
      }
    }
    for (int kb = 0; ok && kb < nk; kb += BATCH) {
      if (kb) load_batch(kb);
      const int kend = min(nk, kb + BATCH);
      if constexpr (LIST) {
        // The batch's groups in the tail buffer (lanes below BATCH: its own
        // units, not the ones looked ahead), outside the loop over stored ones.
#pragma unroll
        for (int s = 0; s < SG; ++s) {
          const bool tail = base[s] >= 0 && base[s] >> a.c.bshift >= newest;
          uint32_t todo = __ballot_sync(0xffffffffu, lane < BATCH && tail);
          while (todo) {
            tail_group(__shfl_sync(0xffffffffu, base[s], __ffs(todo) - 1));
            todo &= todo - 1;
          }
          if (tail) base[s] = -1;  // nothing to stream
        }
      }
      for (; k < kend; ++k) {
        if (k + S - 1 < nk) issue(k + S - 1, kb);  // into the stage unit k - 1 has left
        const uint32_t st = (wseq + k) % S;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[warp][st], ((wseq + k) / S) & 1, tries))) {
          ok = false;
          break;
        }
        const uint32_t stage = wring + st * L::STAGE;
        int at[SG];
        float x[SG][4], vs[SG], gm = kNegInf;
        bool any = false;
#pragma unroll
        for (int s = 0; s < SG; ++s) {
          at[s] = __shfl_sync(0xffffffffu, base[s], k - kb);
          const float ks = __shfl_sync(0xffffffffu, ksc[s], k - kb);
          vs[s] = __shfl_sync(0xffffffffu, vsc[s], k - kb);
          if (at[s] >= 0) {
            any = true;
            float sc[2][4];
            kv8_scores<D, FMT>(stage + s * L::GROUP, qa, sc, lane);
            const float mul = qmul * ks;
            x[s][0] = sc[0][0] * mul; x[s][1] = sc[0][1] * mul;
            x[s][2] = sc[1][0] * mul; x[s][3] = sc[1][1] * mul;
            gm = fmaxf(gm, fmaxf(fmaxf(x[s][0], x[s][1]), fmaxf(x[s][2], x[s][3])) + kv8_exponent(vs[s]));
          } else {
            x[s][0] = x[s][1] = x[s][2] = x[s][3] = kNegInf;
          }
        }
        if (any) {
          const float mref = softmax_step(gm);
          [[maybe_unused]] float entry = 0.f;
#pragma unroll
          for (int s = 0; s < SG; ++s) {
            if (at[s] < 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[s][i] = kv8_ex2(x[s][i] - mref);
            const float psum = (x[s][0] + x[s][1]) + (x[s][2] + x[s][3]);
            l_run += psum;
            const uint32_t p0 = kv8_h2(__floats2half2_rn(x[s][0] * vs[s], x[s][1] * vs[s]));
            const uint32_t p1 = kv8_h2(__floats2half2_rn(x[s][2] * vs[s], x[s][3] * vs[s]));
            kv8_pv<D, FMT>(stage + (SG + s) * L::GROUP, o, p0, p1, lane);
            if constexpr (MASS) {
              // groups that share an entry add up to the entry's last one
              entry += psum;
              if (((at[s] + 16) & ((1 << a.gshift) - 1)) == 0) {
                entry += __shfl_xor_sync(0xffffffffu, entry, 1);
                entry += __shfl_xor_sync(0xffffffffu, entry, 2);
                if (m == 0 && r < G)
                  a.grp[((size_t)row * G + r) * (a.Cap >> a.gshift) + (at[s] >> a.gshift)] = make_float2(entry, mref);
                entry = 0.f;
              }
            }
          }
        }
        // the stage is read before the copy engine may write it again
        __syncwarp();
        if (lane == 0) fence_proxy_async_smem();
      }
    }
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0) {
        note_wait_timeout();
        sh.s_fail = 1;
        // the copies still in flight land before the ring is reused or left
        if (!failed)
          for (int k2 = k; k2 < min(nk, k + S); ++k2)
            mbar_wait(&full[warp][(wseq + k2) % S], ((wseq + k2) / S) & 1, tries);
      }
      // an infinite running max makes this warp's merge weight NaN at every later merge
      m_run = __int_as_float(0x7f800000);
    }
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
    if (m == 0) {
      sM[warp][r] = m_run;
      sL[warp][r] = l_run;
    }
    wseq += failed ? 0u : (uint32_t)nk;
    __syncthreads();  // every warp's stages have been consumed (or drained): the rings become the merge area

    float* sO = reinterpret_cast<float*>(ring);  // [W][8 heads][MROW]
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      const int p = 16 * t + 2 * r;
      *reinterpret_cast<float2*>(sO + (warp * 8 + 2 * m) * L::MROW + p) = make_float2(o[t][0], o[t][2]);
      *reinterpret_cast<float2*>(sO + (warp * 8 + 2 * m + 1) * L::MROW + p) = make_float2(o[t][1], o[t][3]);
    }
    if (threadIdx.x < 8) {
      const int g = threadIdx.x;
      float M = kNegInf, Lh = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, sM[w][g]);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        // a NaN sum without a maximum (every score NaN) is kept
        const float f = sM[w][g] == kNegInf ? (sL[w][g] == 0.f ? 0.f : 1.f) : kv8_ex2(sM[w][g] - M);
        sF[w][g] = f;
        Lh = fmaf(sL[w][g], f, Lh);
      }
      if (Lh != Lh && M == kNegInf) M = 0.f;
      sHm[g] = M;
      sHl[g] = Lh;
    }
    __syncthreads();
    if constexpr (CL) {
      __shared__ Kv8Inbox<D> inbox;
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
        const int g = i / D, d = i % D;
        float M = kNegInf, Lh = 0.f, av = 0.f;
        for (int s = 0; s < C; ++s) M = fmaxf(M, inbox.m[s * 8 + g]);
        for (int s = 0; s < C; ++s) {
          const float ms = inbox.m[s * 8 + g];
          const float f = ms == kNegInf ? 0.f : kv8_ex2(ms - M);
          Lh = fmaf(inbox.l[s * 8 + g], f, Lh);
          av = fmaf(inbox.o[s * chunk + (i - split * chunk)], f, av);
        }
        kv8_finish<D>(a, (size_t)row * G + g, h * G + g, M, Lh, av, kv8_channel<D>(d));
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
        kv8_finish<D>(a, (size_t)row * G + g, h * G + g, sHm[g], sHl[g], av, kv8_channel<D>(d));
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
        // a thread per four channels of a head; the first sixteen contributors'
        // values are in flight while the weights are formed
        static_assert(8 * D / 4 <= NT, "one float4 of the output a thread");
        const int g4 = threadIdx.x / (D / 4), d4 = threadIdx.x % (D / 4);
        auto part = [&](int jj) {
          return jj < n && g4 < G ? __ldcg(reinterpret_cast<const float4*>(a.po + ((size_t)sh.s_slot[jj] * G + g4) * D) + d4)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        constexpr int U = 16, H = kKv8Weights / 32;
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = part(u);
        for (int g = warp; g < G; g += W) {
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
          for (int jj = lane + kKv8Weights; jj < n; jj += 32) M = fmaxf(M, __ldcg(a.pm + (size_t)sh.s_slot[jj] * G + g));
          M = warp_max(M);
          const float sk = a.sink ? a.sink[h * G + g] * kLog2e : kNegInf;
          M = fmaxf(M, sk);
          auto weight = [&](float ms) { return (ms == kNegInf || M == kNegInf) ? 0.f : kv8_ex2(ms - M); };
#pragma unroll
          for (int u = 0; u < H; ++u) {
            const float w = weight(pm[u]);
            Ls += pl[u] * w;
            if (lane + 32 * u < n) sh.s_w[g][lane + 32 * u] = w;
          }
          for (int jj = lane + kKv8Weights; jj < n; jj += 32) {
            const size_t at = (size_t)sh.s_slot[jj] * G + g;
            Ls += __ldcg(a.pl + at) * weight(__ldcg(a.pm + at));
          }
          Ls = warp_sum(Ls);
          if (a.sink && M != kNegInf) Ls += kv8_ex2(sk - M);
          if (lane == 0) {
            const float inv = Ls == 0.f ? 0.f : 1.f / Ls;  // NaN stays NaN
            const size_t hq = (size_t)row * G + g;
            sh.s_m[g] = M;
            sh.s_inv[g] = inv;
            if (a.lse) a.lse[hq] = Ls == 0.f ? kNegInf : M * kLn2 + logf(Ls);
            if (a.fin) a.fin[hq] = make_float2(M, inv);
          }
        }
        __syncthreads();
        if (g4 < G) {
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int j0 = 0; j0 < n; j0 += U) {
            if (j0)
#pragma unroll
              for (int u = 0; u < U; ++u) v[u] = part(j0 + u);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int jj = j0 + u;
              if (jj >= n) break;
              float w;
              if (jj < kKv8Weights) {
                w = sh.s_w[g4][jj];
              } else {
                const float ms = __ldcg(a.pm + (size_t)sh.s_slot[jj] * G + g4);
                w = (ms == kNegInf || sh.s_m[g4] == kNegInf) ? 0.f : kv8_ex2(ms - sh.s_m[g4]);
              }
              acc.x = fmaf(v[u].x, w, acc.x);
              acc.y = fmaf(v[u].y, w, acc.y);
              acc.z = fmaf(v[u].z, w, acc.z);
              acc.w = fmaf(v[u].w, w, acc.w);
            }
          }
          const float inv = sh.s_inv[g4];
          bf16* op = a.out + ((size_t)row * G + g4) * D;
          *reinterpret_cast<__nv_bfloat162*>(op + kv8_channel<D>(4 * d4)) = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
          *reinterpret_cast<__nv_bfloat162*>(op + kv8_channel<D>(4 * d4 + 2)) =
              __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
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

// mass_out = mass_in + the blocks' weight sums: a lane per entry of each head's
// sums (coalesced loads, all heads' in flight together), the entries of a block
// added by shuffles in a fixed order.
__global__ void __launch_bounds__(256)
kv8_mass_kernel(const Kv8Attend a, int per_row) {
  pdl_wait_then_release();
  const int row = blockIdx.x / per_row, at = (blockIdx.x % per_row) * 256 + threadIdx.x;
  const int eshift = a.c.bshift - a.gshift, blk = at >> eshift;  // 2^eshift <= 16 entries per block
  const bool live = blk < clamp_len(a.ctx_len[row / a.Hkv], a.Cap) >> a.c.bshift;
  float sum = 0.f;
  if (live) {
    float2 x[8], f[8];
#pragma unroll
    for (int g = 0; g < 8; ++g)
      if (g < a.G) {
        x[g] = __ldcg(a.grp + ((size_t)row * a.G + g) * (a.Cap >> a.gshift) + at);
        f[g] = a.fin[(size_t)row * a.G + g];
      }
#pragma unroll
    for (int g = 0; g < 8; ++g)
      if (g < a.G) sum += x[g].x * kv8_ex2(x[g].y - f[g].x) * f[g].y;
  }
  for (int o = 1; o < (1 << eshift); o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (live && (at & ((1 << eshift) - 1)) == 0) {
    const size_t b = (size_t)row * (a.Cap >> a.c.bshift) + blk;
    a.mass_out[b] = (a.mass_in ? a.mass_in[b] : 0.f) + sum;
  }
}

// ------------------------------------------------------------------- launches

// The driver's tensor-map encoder, looked up once.
static PFN_cuTensorMapEncodeTiled_v12000 kv8_encode_fn() {
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

// Codes as [rows * Cap] rows of D bytes, boxes of `box_rows` whole rows.
static bool kv8_map(CUtensorMap* map, const void* base, uint64_t rows, int D, int box_rows) {
  auto fn = kv8_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)D};
  cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Twelve warps (at most 170 registers a thread) whose rings of two 32-token
// units fill the shared memory: 8, 10, 14 and 16 warps and units of 16 tokens
// were slower.  At D = 64 int8 units of 64 tokens (half the softmax steps)
// are 9% faster, but 7% slower for e4m3, whose conversions are the longer chain.
template <int D, int FMT>
struct Kv8Config {
  static constexpr int SG = D == 64 && FMT == kKv8Int8 ? 4 : 2, W = 12, S = D == 128 || SG == 4 ? 2 : 4;
  using L = Kv8Layout<D, SG, W, S>;
  static constexpr size_t smem(int rows) { return L::REGION + (size_t)(rows + 1) * sizeof(int) + 1024; }
};

bool kv8_attend_supported(const Shape& s) {
  return s.dtype == 1 && s.B * (long long)s.Hkv <= kKv8MaxRows && (long long)s.B * s.Hkv * s.Cap < (1ll << 31);
}

static int kv8_grid() { return std::min(sm_count() * kKv8PerSm, kKv8MaxGrid); }
static size_t a256(size_t v) { return (v + 255) & ~(size_t)255; }

// log2 of the tokens of one entry of the weight sums (a unit of the kernel that runs,
// or a block if that is smaller).
static int kv8_entry_shift(const Shape& s, const Kv8& c) {
  const int unit = 16 * (s.D == 128 ? (c.format == kKv8Int8 ? Kv8Config<128, kKv8Int8>::SG : Kv8Config<128, kKv8E4m3>::SG)
                                    : (c.format == kKv8Int8 ? Kv8Config<64, kKv8Int8>::SG : Kv8Config<64, kKv8E4m3>::SG));
  return __builtin_ctz((unsigned)std::min(unit, c.block));
}

size_t kv8_attend_workspace(const Shape& s, const Kv8& c, bool with_mass) {
  const size_t rows = (size_t)s.B * s.Hkv, slots = 2 * (size_t)kv8_grid();
  return kKv8TicketBytes + a256(slots * s.G * s.D * 4) + 2 * a256(slots * s.G * 4) +
         (with_mass ? a256(rows * s.G * 8) + a256(rows * s.G * (s.Cap >> kv8_entry_shift(s, c)) * 8) : 0);
}

// What a launch of one kernel needs once per device: the limit of its dynamic
// shared memory raised, and the number of clusters of each size that fit.
struct Kv8Device {
  std::atomic<int> clusters[kKv8MaxCluster + 1];  // 0: not asked yet, else 1 + the number
  std::atomic<bool> raised;
};

template <int D, int FMT, bool LIST, bool MASS, bool CL>
static cudaError_t kv8_prepare(Kv8Device** out) {
  using F = Kv8Config<D, FMT>;
  static Kv8Device devices[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  Kv8Device& d = devices[dev];
  if (!d.raised.load(std::memory_order_acquire)) {
    auto kern = kv8_attend_kernel<D, FMT, F::SG, F::W, F::S, LIST, MASS, CL>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F::smem(CL ? 0 : kKv8MaxRows));
    if (e == cudaSuccess && CL) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    d.raised.store(true, std::memory_order_release);
  }
  *out = &d;
  return cudaSuccess;
}

// Clusters of c CTAs of the cluster kernel that run at once (asked once per device).
template <int D, int FMT, bool LIST, bool MASS>
static int kv8_clusters(int c, Kv8Device* d) {
  using F = Kv8Config<D, FMT>;
  int n = d->clusters[c].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(F::W * 32);
    cfg.dynamicSmemBytes = F::smem(0);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int got = 0;
    auto kern = kv8_attend_kernel<D, FMT, F::SG, F::W, F::S, LIST, MASS, true>;
    if (cudaOccupancyMaxActiveClusters(&got, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      got = 0;
    }
    n = 1 + got;
    d->clusters[c].store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

// CTAs per row of the cluster kernel, or 0 for ranges over all rows: whichever the
// measured costs make faster.  A CTA takes t ns a token (4.9 at D = 128, 2.7 at
// D = 64) and a cluster 5.5 us besides, in as many waves as the clusters need; the
// ranges take 13 us, 6 per row beyond their equal shares, and 0.1 for each CTA that shares
// a row.  Measured on 50 shapes of 1 to 256 rows, full but for a tenth, of 1k to 64k tokens,
// both sides each: 27.5 us with a CTA a row and 30.3 in ranges for 96 rows of 4k at D = 128,
// 76 and 66 at 16k; 28.9 with two a row and 32.8 for 64 rows of 16k at D = 64, 94 and 87 at
// 64k.  Where it takes the slower side it loses 9% at most (256 rows of 4k at D = 128: 57.9
// us against 53.0).
// `most` bounds a row's tokens; where only the device knows them, rows are taken to hold three quarters
// of it on average and a cluster to wait for one that is full.
template <int D, int FMT, bool LIST, bool MASS>
static int kv8_pick(int rows, double most, bool fixed, bool even, Kv8Device* d) {
  const double t = D == 128 ? 4.9e-3 : 2.7e-3, sms = sm_count();
  const double mean = fixed ? most : 0.75 * most, longest = even ? mean : most;
  double best = 13.0 + rows / sms * (mean * t + 6.0) + 0.1 * sms / rows;
  int pick = 0;
  for (int c = 1; c <= kKv8MaxCluster; ++c) {
    const int n = c == 1 ? sm_count() : kv8_clusters<D, FMT, LIST, MASS>(c, d);
    if (n < 1) continue;
    const double us = ((rows + n - 1) / n) * (5.5 + longest / c * t);
    if (us < best) {
      best = us;
      pick = c;
    }
  }
  return pick;
}

template <int D, int FMT, bool LIST, bool MASS>
static cudaError_t kv8_launch(Kv8Attend a, cudaStream_t st) {
  using F = Kv8Config<D, FMT>;
  constexpr int SG = F::SG, W = F::W, S = F::S;
  a.boxes = LIST && a.P < 16 * SG ? SG : 1;
  CUtensorMap tk, tv;
  const uint64_t tokens = (uint64_t)a.rows * a.Cap;
  if (!kv8_map(&tk, a.c.kc, tokens, D, 16 * SG / a.boxes) || !kv8_map(&tv, a.c.vc, tokens, D, 16 * SG / a.boxes))
    return cudaErrorInvalidValue;
  Kv8Device* d;
  cudaError_t e = kv8_prepare<D, FMT, LIST, MASS, true>(&d);
  if (e != cudaSuccess) return e;
  const bool fixed = LIST && !a.count;  // lists of one length; one sequence's rows are of one length too
  const double most = LIST ? (double)(a.count ? a.idx_stride : a.k_fixed) * a.P : a.Cap;
  a.cluster = kv8_pick<D, FMT, LIST, MASS>(a.rows, most, fixed, fixed || (!LIST && a.rows == a.Hkv), d);
  if (a.cluster)
    return launch_pdl_cluster(kv8_attend_kernel<D, FMT, SG, W, S, LIST, MASS, true>, dim3(a.rows * a.cluster),
                              dim3(W * 32), F::smem(0), a.cluster, st, tk, tv, a);
  if ((e = kv8_prepare<D, FMT, LIST, MASS, false>(&d)) != cudaSuccess) return e;
  return launch_pdl(kv8_attend_kernel<D, FMT, SG, W, S, LIST, MASS, false>, dim3(kv8_grid()), dim3(W * 32),
                    F::smem(a.rows), st, tk, tv, a);
}

template <int D>
static cudaError_t kv8_dispatch(const Kv8Attend& a, cudaStream_t st) {
  if (a.page_idx)
    return a.c.format == kKv8Int8 ? kv8_launch<D, kKv8Int8, true, false>(a, st) : kv8_launch<D, kKv8E4m3, true, false>(a, st);
  if (a.mass_out)
    return a.c.format == kKv8Int8 ? kv8_launch<D, kKv8Int8, false, true>(a, st) : kv8_launch<D, kKv8E4m3, false, true>(a, st);
  return a.c.format == kKv8Int8 ? kv8_launch<D, kKv8Int8, false, false>(a, st) : kv8_launch<D, kKv8E4m3, false, false>(a, st);
}

cudaError_t launch_kv8_attend(const Shape& s, const Kv8& c, const void* q, const int32_t* page_idx, int idx_stride,
                              const int32_t* count, int k_fixed, const int32_t* ctx_len, const float* sink,
                              void* out, float* lse, const float* mass_in, float* mass_out, void* ws,
                              cudaStream_t st) {
  Kv8Attend a = {};
  a.c = c;
  a.q = static_cast<const bf16*>(q);
  a.page_idx = page_idx;
  a.count = count;
  a.ctx_len = ctx_len;
  a.idx_stride = idx_stride;
  a.k_fixed = k_fixed;
  a.rows = s.B * s.Hkv;
  a.Hq = s.Hq; a.Hkv = s.Hkv; a.G = s.G; a.Cap = s.Cap; a.P = s.P; a.pshift = s.pshift;
  a.test_wait = (s.flags & kFlagTestWaitTimeout) ? 1 : 0;
  a.qscale = s.scale * kLog2e;
  a.sink = sink;
  a.out = static_cast<bf16*>(out);
  a.lse = lse;
  const size_t rows = (size_t)a.rows, slots = 2 * (size_t)kv8_grid();
  char* w = static_cast<char*>(ws);
  auto take = [&](size_t bytes) {
    char* p = w;
    w += a256(bytes);
    return p;
  };
  a.tickets = reinterpret_cast<int32_t*>(take(kKv8TicketBytes));
  a.po = reinterpret_cast<float*>(take(slots * s.G * s.D * 4));
  a.pm = reinterpret_cast<float*>(take(slots * s.G * 4));
  a.pl = reinterpret_cast<float*>(take(slots * s.G * 4));
  if (mass_out) {
    a.fin = reinterpret_cast<float2*>(take(rows * s.G * 8));
    a.gshift = kv8_entry_shift(s, c);
    a.grp = reinterpret_cast<float2*>(take(rows * s.G * (s.Cap >> a.gshift) * 8));
    a.mass_in = mass_in;
    a.mass_out = mass_out;
  }
  cudaError_t e = s.D == 64 ? kv8_dispatch<64>(a, st) : kv8_dispatch<128>(a, st);
  if (e == cudaSuccess && mass_out) {
    const int per_row = ((s.Cap >> a.gshift) + 255) / 256;
    e = launch_pdl(kv8_mass_kernel, dim3((unsigned)a.rows * per_row), dim3(256), 0, st, a, per_row);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

DeviceStatus take_status_attend_kv8() { return take_status_here(); }

}  // namespace sls
