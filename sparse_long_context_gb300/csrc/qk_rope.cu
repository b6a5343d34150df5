// Per-head root-mean-square norm of queries and keys and the rotation by the
// token's position in one pass over the projected heads:
//   y = x w / sqrt(mean(x^2) + eps),  (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin).
// Bound by memory: every element is read and written once.  32768 tokens of 28 + 4
// heads of 128 channels take 91 us (5.9 TB/s, 87% of the measured copy), 16384 in
// fp32 with half of the channels rotated 86 us (92%), 1000 tokens 6.2 us, 32 tokens of
// 12 + 2 heads 1.8 us, the launch.  Tokens of few heads are bound by the sines and
// coefficients, which are a token's whatever its heads: 16384 tokens of 8 + 1 heads 20 us
// (floor 11), 23029 of 7 + 1 heads of 64 channels 10.7 (floor 7).  (Times of the device
// alone, calls replayed from a graph.)  The arithmetic is fp32 throughout, the norm's
// reciprocal root within 2 ulp; the one rounding to fewer bits is the output's.
//
// A lane holds two 16-byte vectors of a head whose channels form whole pairs (vector
// l and vector R/2 further on when halves are paired), so a pair never leaves the
// lane; at D = 128 in bf16 a head is 8 lanes and a warp takes 4 heads at a time.  With
// the norm's weights the rotation of a pair is
//   y_a = inv (x_a w_a cos - x_b w_b sin),  y_b = inv (x_b w_b cos + x_a w_a sin),
// whose four products of weight, cosine and sine are formed once per token for all
// of its query heads and once for its key heads; channels that are not rotated
// have cos = 1, sin = 0.  Issue slots come next after memory, so the arithmetic is
// in two-float instructions and the sines are shared by the lanes that need the same.
// The loads of four steps are in flight together.  Measured against it: vectors of 8
// bytes (half as wide steps; 90 us on the bf16 prompt, but 7.8 on 1000 tokens and 95 in
// fp32), rings of asynchronous copies (115) and of registers (109), L2 prefetches of the
// next token (110).
//
// Angles are kept in turns: positions[t] * f_i modulo one turn is the low 64
// bits of the product with the frequency as a 64-bit fixed-point fraction
// (one turn = 2^64), exact for every position, so only the frequency's own
// rounding (2^-56 turns) is multiplied by the position.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace sls {

constexpr int kRopeThreads = 128, kRopePerSm = 4;  // more CTAs per SM spill: 118 us at 7
constexpr int kRopeOnePerSm = 5;  // of the kernel of single steps (4 and 6: 7% and 10% to 38% slower)
constexpr int kRopeUnroll = 4;  // warp steps whose loads are in flight together

// A 16-byte vector, not kept in L1 (plain loads: the outputs may be the inputs).
__device__ __forceinline__ uint4 rope_load(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// A vector of weights, which stays in L1.  Loaded at each token: 16 registers a side
// that hold them for all tokens spill (97 us on the bf16 prompt).
__device__ __forceinline__ uint4 rope_weights(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Two floats in one 64-bit register: products and sums of both at once.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_split(F2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 f2_swap(F2 v) {
  float a, b;
  f2_split(v, a, b);
  return f2(b, a);
}

__device__ __forceinline__ void rope_unpack(const float*, uint4 v, F2 (&x)[2]) {
  x[0] = f2(__uint_as_float(v.x), __uint_as_float(v.y));
  x[1] = f2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void rope_unpack(const bf16*, uint4 v, F2 (&x)[4]) {
  x[0] = f2(bf16lo(v.x), bf16hi(v.x));
  x[1] = f2(bf16lo(v.y), bf16hi(v.y));
  x[2] = f2(bf16lo(v.z), bf16hi(v.z));
  x[3] = f2(bf16lo(v.w), bf16hi(v.w));
}
__device__ __forceinline__ void rope_store(float* p, const F2 (&x)[2]) {
  float4 y;
  f2_split(x[0], y.x, y.y);
  f2_split(x[1], y.z, y.w);
  *reinterpret_cast<float4*>(p) = y;
}
__device__ __forceinline__ void rope_store(bf16* p, const F2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f2_split(x[i], a, b);
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// What one side's heads are multiplied by for a token.  The lane's channels are
// two vectors x and z of 2 NF, in float pairs, and
//   paired halves:  y = x A + z B,  v = z C + x E        (pair i: x_i with z_i)
//   interleaved:    y = x A + swap(x) B,  v = z C + swap(z) E
template <int NF>
struct RopeCoef {
  F2 A[NF], B[NF], C[NF], E[NF];
};
template <typename T, bool INTER, int NF>
__device__ __forceinline__ void rope_coef(RopeCoef<NF>& r, const T* w, int c0, int c1, const float (&cs)[2 * NF],
                                          const float (&sn)[2 * NF]) {
  float wx[2 * NF], wz[2 * NF];
  if (w) {
    F2 a[NF], b[NF];
    rope_unpack(w, rope_weights(w + c0), a);
    rope_unpack(w, rope_weights(w + c1), b);
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      f2_split(a[i], wx[2 * i], wx[2 * i + 1]);
      f2_split(b[i], wz[2 * i], wz[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * NF; ++i) wx[i] = wz[i] = 1.f;
  }
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    const int a = 2 * i, b = a + 1;
    if constexpr (INTER) {  // angle i turns pair (a, b) of x, angle NF + i that of z
      r.A[i] = f2(wx[a] * cs[i], wx[b] * cs[i]);
      r.B[i] = f2(-wx[b] * sn[i], wx[a] * sn[i]);
      r.C[i] = f2(wz[a] * cs[NF + i], wz[b] * cs[NF + i]);
      r.E[i] = f2(-wz[b] * sn[NF + i], wz[a] * sn[NF + i]);
    } else {
      r.A[i] = f2(wx[a] * cs[a], wx[b] * cs[b]);
      r.B[i] = f2(-wz[a] * sn[a], -wz[b] * sn[b]);
      r.C[i] = f2(wz[a] * cs[a], wz[b] * cs[b]);
      r.E[i] = f2(wx[a] * sn[a], wx[b] * sn[b]);
    }
  }
}

// The lanes of a head, and the heads of a warp step.
template <typename T, int D>
struct RopeShape {
  static constexpr int VC = 16 / sizeof(T);  // channels of a vector
  static constexpr int L = D / (2 * VC), HS = 32 / L;
  static constexpr int PER = VC / HS > 1 ? VC / HS : 1;  // angles whose sines a lane forms
};

// The coefficients of one side for a token, from the sines that the warp's lanes formed.
template <typename T, int D, bool INTER, bool FULL>
__device__ __forceinline__ void rope_side_coef(RopeCoef<RopeShape<T, D>::VC / 2>& k, const T* w, int c0, int c1,
                                               const float (&mc)[RopeShape<T, D>::PER],
                                               const float (&ms)[RopeShape<T, D>::PER], bool rot) {
  using S = RopeShape<T, D>;
  float cs[S::VC], sn[S::VC];
#pragma unroll
  for (int i = 0; i < S::VC; ++i) {
    cs[i] = __shfl_sync(0xffffffffu, mc[i % S::PER], (i / S::PER) * S::L + (threadIdx.x & 31) % S::L);
    sn[i] = __shfl_sync(0xffffffffu, ms[i % S::PER], (i / S::PER) * S::L + (threadIdx.x & 31) % S::L);
  }
  rope_coef<T, INTER, S::VC / 2>(k, w, c0, c1, cs, sn);
  if (!FULL && !rot) {  // sin = 0, but an infinite weight times it is not
#pragma unroll
    for (int i = 0; i < S::VC / 2; ++i) k.B[i] = k.E[i] = 0ull;
  }
}

// One step: the lane's two vectors of a head, normalised (`norm` for the warp, `mine` for
// the lane's head), rotated and stored (if `live`).
template <typename T, int D, bool INTER, bool FULL>
__device__ __forceinline__ void rope_step(T* out, uint4 r0, uint4 r1, const RopeCoef<RopeShape<T, D>::VC / 2>& k, bool norm,
                                          int c0, int c1, float eps, bool rot, bool live, bool mine = true) {
  constexpr int L = RopeShape<T, D>::L, NF = RopeShape<T, D>::VC / 2;
  F2 x[NF], z[NF];
  rope_unpack(out, r0, x);
  rope_unpack(out, r1, z);
  float inv = 1.f;
  if (norm) {
    F2 q = f2_mul(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < NF; ++i) q = f2_fma(x[i], x[i], q);
#pragma unroll
    for (int i = 0; i < NF; ++i) q = f2_fma(z[i], z[i], q);
    float ss, hi;
    f2_split(q, ss, hi);
    ss += hi;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    inv = mine ? rsqrtf(ss * (1.f / D) + eps) : 1.f;
  }
  const F2 iv = f2(inv, inv);
  F2 y[NF], v[NF];
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    // channels that are not rotated do not see their neighbour (0 * inf)
    const F2 xo = INTER ? f2_swap(x[i]) : z[i], zo = INTER ? f2_swap(z[i]) : x[i];
    y[i] = f2_mul(f2_fma(FULL || rot ? xo : 0ull, k.B[i], f2_mul(x[i], k.A[i])), iv);
    v[i] = f2_mul(f2_fma(FULL || rot ? zo : 0ull, k.E[i], f2_mul(z[i], k.C[i])), iv);
  }
  if (live) {
    rope_store(out + c0, y);
    rope_store(out + c1, v);
  }
}

// Steps [s0, s1) of one side (queries or keys) of a token: step s holds heads
// s HS .. s HS + HS - 1.  FULL: every channel is rotated.
template <typename T, int D, bool INTER, bool FULL>
__device__ __forceinline__ void rope_side(const T* in, int64_t in_h, T* out, int64_t out_h, const T* w, int heads, int s0,
                                          int s1, int c0, int c1, const float (&mc)[RopeShape<T, D>::PER],
                                          const float (&ms)[RopeShape<T, D>::PER], float eps, int sub, bool rot) {
  constexpr int HS = RopeShape<T, D>::HS, U = kRopeUnroll;
  RopeCoef<RopeShape<T, D>::VC / 2> k;
  rope_side_coef<T, D, INTER, FULL>(k, w, c0, c1, mc, ms, rot);
  int h = s0 * HS + sub;
  const int hend = min(heads, s1 * HS);
  in += h * in_h;
  out += h * out_h;
  in_h *= HS;
  out_h *= HS;
  for (int s = s0; s < s1; s += U) {
    uint4 r0[U], r1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r0[u] = r1[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h + u * HS < hend) {
        r0[u] = rope_load(in + c0);
        r1[u] = rope_load(in + c1);
      }
      in += in_h;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u < s1)
        rope_step<T, D, INTER, FULL>(out, r0[u], r1[u], k, w != nullptr, c0, c1, eps, rot, h + u * HS < hend);
      out += out_h;
    }
    h += U * HS;
  }
}

// A warp takes items (a token, or one of its `chunks` shares of `per` steps).  The
// lanes that hold the same channels of the warp's HS heads share the sines'
// work: each forms VC / HS (at least one) of the VC angles' and hands them on.
// FEW: all steps of a token's two sides fit in one group of kRopeUnroll.  Their loads go
// out together before the sines, and the next token's position before that, so a
// token waits for memory once and not three times: 16384 tokens of 8 + 1 heads of 128
// 25.0 -> 19.8 us.
template <typename T, int D, bool INTER, bool FULL, bool FEW>
__global__ void __launch_bounds__(kRopeThreads, kRopePerSm)
qk_norm_rope_kernel(const __grid_constant__ RopeArgs a, int per, int chunks) {
  using S = RopeShape<T, D>;
  constexpr int VC = S::VC, L = S::L, HS = S::HS, PER = S::PER;
  const int lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
  const int half = FULL ? D / 2 : a.R >> 1;
  const bool rot = FULL || 2 * VC * l < a.R;  // R is a multiple of 16: a lane is rotated whole or not at all
  const int c0 = INTER || !rot ? 2 * VC * l : VC * l, c1 = INTER || !rot ? c0 + VC : half + VC * l;
  uint64_t f[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = rot ? a.freq[VC * l + (sub * PER + i) % VC] : 0ull;
  const int qsteps = (a.Hq + HS - 1) / HS, steps = qsteps + (a.Hkv + HS - 1) / HS;
  pdl_wait_then_release();
  const int64_t warps = (int64_t)gridDim.x * (kRopeThreads / 32), items = (int64_t)a.N * chunks;
  int64_t it = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  int next = FEW && it < items ? a.pos[it] : 0;
  for (; it < items; it += warps) {
    const int64_t t = chunks == 1 ? it : it / chunks;
    const int s0 = chunks == 1 ? 0 : (int)(it - t * chunks) * per, s1 = min(s0 + per, steps);
    const int pos = FEW ? next : a.pos[t];
    if (FEW && it + warps < items) next = a.pos[it + warps];
    if (pos < 0) continue;
    const T* qi = static_cast<const T*>(a.q) + t * a.q_t;
    const T* ki = static_cast<const T*>(a.k) + t * a.k_t;
    T* qo = static_cast<T*>(a.qo) + t * a.qo_t;
    T* ko = static_cast<T*>(a.ko) + t * a.ko_t;
    uint4 r0[kRopeUnroll], r1[kRopeUnroll];
    if constexpr (FEW) {
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const bool key = u >= qsteps;
        const int h = (key ? u - qsteps : u) * HS + sub;
        r0[u] = r1[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < (key ? a.Hkv : a.Hq)) {
          const T* in = key ? ki + h * a.k_h : qi + h * a.q_h;
          r0[u] = rope_load(in + c0);
          r1[u] = rope_load(in + c1);
        }
      }
    }
    float mc[PER], ms[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t turn = (int64_t)((uint64_t)(int64_t)pos * f[i]);
      sincospif((float)turn * 1.0842021724855044e-19f, &ms[i], &mc[i]);  // 2^-63: half turns in [-1, 1]
    }
    if constexpr (FEW) {
      RopeCoef<VC / 2> k;
      if (qsteps) {
        rope_side_coef<T, D, INTER, FULL>(k, static_cast<const T*>(a.wq), c0, c1, mc, ms, rot);
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u)
          if (u < qsteps)
            rope_step<T, D, INTER, FULL>(qo + (u * HS + sub) * a.qo_h, r0[u], r1[u], k, a.wq != nullptr, c0, c1, a.eps, rot,
                                         u * HS + sub < a.Hq);
      }
      if (steps > qsteps) {
        rope_side_coef<T, D, INTER, FULL>(k, static_cast<const T*>(a.wk), c0, c1, mc, ms, rot);
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u)
          if (u >= qsteps && u < steps) {
            const int h = (u - qsteps) * HS + sub;
            rope_step<T, D, INTER, FULL>(ko + h * a.ko_h, r0[u], r1[u], k, a.wk != nullptr, c0, c1, a.eps, rot, h < a.Hkv);
          }
      }
    } else {
      if (s0 < qsteps)
        rope_side<T, D, INTER, FULL>(qi, a.q_h, qo, a.qo_h, static_cast<const T*>(a.wq), a.Hq, s0, min(s1, qsteps), c0, c1,
                                     mc, ms, a.eps, sub, rot);
      if (s1 > qsteps)
        rope_side<T, D, INTER, FULL>(ki, a.k_h, ko, a.ko_h, static_cast<const T*>(a.wk), a.Hkv, max(s0 - qsteps, 0),
                                     s1 - qsteps, c0, c1, mc, ms, a.eps, sub, rot);
    }
  }
}

// A warp step by itself: heads are numbered through queries and keys, and a lane keeps
// to its head's side.  steps == 1: a token's heads are one step.  A warp takes tokens in
// turn, with the next one's vectors and the position of the one after in flight: 23029
// tokens of 7 + 1 heads of 64 channels 19.9 -> 10.6 us, 32484 of 3 + 1 of 128 30.8 -> 14.9.
// steps > 1: few tokens, a warp each for every step, whose vectors are loaded together
// with the position: 32 tokens of 12 + 2 heads 2.8 -> 1.8 us, 370 of 28 + 4 3.9 -> 3.4.
template <typename T, int D, bool INTER, bool FULL>
__global__ void __launch_bounds__(kRopeThreads, kRopeOnePerSm)
qk_norm_rope_one_kernel(const __grid_constant__ RopeArgs a, int steps) {
  using S = RopeShape<T, D>;
  constexpr int VC = S::VC, L = S::L, HS = S::HS, PER = S::PER;
  const int lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
  const int half = FULL ? D / 2 : a.R >> 1;
  const bool rot = FULL || 2 * VC * l < a.R;
  const int c0 = INTER || !rot ? 2 * VC * l : VC * l, c1 = INTER || !rot ? c0 + VC : half + VC * l;
  uint64_t f[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = rot ? a.freq[VC * l + (sub * PER + i) % VC] : 0ull;
  int64_t t = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5), stride = (int64_t)gridDim.x * (kRopeThreads / 32);
  int h = sub;
  if (steps > 1) {
    h += (int)(t % steps) * HS;
    t /= steps;
    stride = a.N;
  }
  if (t >= a.N) return;
  const bool key = h >= a.Hq, live = h < a.Hq + a.Hkv;
  h -= key ? a.Hq : 0;
  const T* in = static_cast<const T*>(key ? a.k : a.q) + h * (key ? a.k_h : a.q_h);
  T* out = static_cast<T*>(key ? a.ko : a.qo) + h * (key ? a.ko_h : a.qo_h);
  const int64_t in_t = key ? a.k_t : a.q_t, out_t = key ? a.ko_t : a.qo_t;
  const T* w = static_cast<const T*>(key ? (a.Hkv ? a.wk : nullptr) : a.wq);
  const bool norm = (a.Hq && a.wq) || (a.Hkv && a.wk);
  pdl_wait_then_release();
  int pos = a.pos[t], next = t + stride < a.N ? a.pos[t + stride] : 0;
  uint4 r0 = make_uint4(0u, 0u, 0u, 0u), r1 = r0, n0 = r0, n1 = r0;
  if (live) {
    r0 = rope_load(in + t * in_t + c0);
    r1 = rope_load(in + t * in_t + c1);
  }
  for (; t < a.N; t += stride) {
    const int64_t t1 = t + stride;
    if (live && t1 < a.N) {
      n0 = rope_load(in + t1 * in_t + c0);
      n1 = rope_load(in + t1 * in_t + c1);
    }
    const int after = t1 + stride < a.N ? a.pos[t1 + stride] : 0;
    if (pos >= 0) {
      float mc[PER], ms[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int64_t turn = (int64_t)((uint64_t)(int64_t)pos * f[i]);
        sincospif((float)turn * 1.0842021724855044e-19f, &ms[i], &mc[i]);  // 2^-63: half turns in [-1, 1]
      }
      RopeCoef<VC / 2> k;
      rope_side_coef<T, D, INTER, FULL>(k, w, c0, c1, mc, ms, rot);
      rope_step<T, D, INTER, FULL>(out + t * out_t, r0, r1, k, norm, c0, c1, a.eps, rot, live, w != nullptr);
    }
    pos = next;
    next = after;
    r0 = n0;
    r1 = n1;
  }
}

template <typename T, int D, bool INTER>
static cudaError_t rope_launch(const RopeArgs& a, cudaStream_t st) {
  constexpr int HS = RopeShape<T, D>::HS, NW = kRopeThreads / 32;
  const int steps = (a.Hq + HS - 1) / HS + (a.Hkv + HS - 1) / HS;
  const int64_t sms = sm_count();
  const int one = (a.Hq + a.Hkv + HS - 1) / HS;
  // steps by themselves while they fit in one wave (500 tokens of 8 steps: 5.0 us against 4.3)
  if (one == 1 || (int64_t)a.N * one <= sms * NW * kRopeOnePerSm) {
    const int64_t ctas = ((int64_t)a.N * one + NW - 1) / NW;
    const dim3 grid((unsigned)(one == 1 ? std::min(ctas, sms * kRopeOnePerSm) : ctas)), block(kRopeThreads);
    const cudaError_t e = a.R == D ? launch_pdl(qk_norm_rope_one_kernel<T, D, INTER, true>, grid, block, 0, st, a, one)
                                   : launch_pdl(qk_norm_rope_one_kernel<T, D, INTER, false>, grid, block, 0, st, a, one);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  // up to a few hundred tokens: a token's heads go to several warps, up to 8 warps per SM
  const int64_t want = std::min<int64_t>(steps, std::max<int64_t>(1, sms * 8 / a.N));
  const int per = (int)((steps + want - 1) / want), chunks = (steps + per - 1) / per;
  const int64_t ctas = std::min<int64_t>(((int64_t)a.N * chunks + NW - 1) / NW, sms * kRopePerSm);
  const dim3 grid((unsigned)ctas), block(kRopeThreads);
  const bool few = chunks == 1 && steps <= kRopeUnroll;
  cudaError_t e;
  if (a.R == D)
    e = few ? launch_pdl(qk_norm_rope_kernel<T, D, INTER, true, true>, grid, block, 0, st, a, per, chunks)
            : launch_pdl(qk_norm_rope_kernel<T, D, INTER, true, false>, grid, block, 0, st, a, per, chunks);
  else
    e = few ? launch_pdl(qk_norm_rope_kernel<T, D, INTER, false, true>, grid, block, 0, st, a, per, chunks)
            : launch_pdl(qk_norm_rope_kernel<T, D, INTER, false, false>, grid, block, 0, st, a, per, chunks);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.dtype == 0) {
    if (a.D == 64) return a.interleaved ? rope_launch<float, 64, true>(a, st) : rope_launch<float, 64, false>(a, st);
    return a.interleaved ? rope_launch<float, 128, true>(a, st) : rope_launch<float, 128, false>(a, st);
  }
  if (a.D == 64) return a.interleaved ? rope_launch<bf16, 64, true>(a, st) : rope_launch<bf16, 64, false>(a, st);
  return a.interleaved ? rope_launch<bf16, 128, true>(a, st) : rope_launch<bf16, 128, false>(a, st);
}

}  // namespace sls
