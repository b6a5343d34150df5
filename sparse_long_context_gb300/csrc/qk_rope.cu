// Per-head root-mean-square norm of queries and keys and the rotation by the
// token's position in one pass over the projected heads:
//   y = x w / sqrt(mean(x^2) + eps),  (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin).
// Bound by memory: every element is read and written once.  32768 tokens of 28 + 4
// heads of 128 channels take 90 us (5.95 TB/s, 88% of the measured copy); 32
// tokens of 12 + 2 heads 3 us, the launch.  Rings of asynchronous copies or of
// registers in place of the plain loads were slower (115 and 109 us): what is
// in flight was enough, resident warps were not.
//
// A head is D/8 lanes of eight channels each, so a warp takes 256 / D heads at a
// time.  A lane's channels are two vectors of four that form whole pairs (channels
// 4l and R/2 + 4l when halves are paired), so a pair never leaves the lane and a
// lane needs four angles.  With the norm's weights the rotation of a pair is
//   y_a = inv (x_a w_a cos - x_b w_b sin),  y_b = inv (x_b w_b cos + x_a w_a sin),
// whose four products of weight, cosine and sine are formed once per token for all
// of its query heads and once for its key heads; channels that are not rotated
// have cos = 1, sin = 0.  Issue slots come next after memory, so the arithmetic is
// in two-float instructions.  The loads of four steps are in flight together.
//
// Angles are kept in turns: positions[t] * f_i modulo one turn is the low 64
// bits of the product with the frequency as a 64-bit fixed-point fraction
// (one turn = 2^64), exact for every position, so only the frequency's own
// rounding (2^-56 turns) is multiplied by the position.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace sls {

constexpr int kRopeThreads = 128, kRopePerSm = 7;  // 4 to 8 CTAs per SM: 100 to 90 us on 32768 tokens
constexpr int kRopeUnroll = 4;  // warp steps whose loads are in flight together

template <typename T> struct Vec4;
template <> struct Vec4<float> { using type = uint4; };
template <> struct Vec4<bf16> { using type = uint2; };

// Four channels, not kept in L1 (plain loads: the outputs may be the inputs).
__device__ __forceinline__ uint4 rope_load(const float* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 rope_load(const bf16* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
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

__device__ __forceinline__ void rope_unpack(uint4 v, F2& a, F2& b) {
  a = f2(__uint_as_float(v.x), __uint_as_float(v.y));
  b = f2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void rope_unpack(uint2 v, F2& a, F2& b) {
  a = f2(bf16lo(v.x), bf16hi(v.x));
  b = f2(bf16lo(v.y), bf16hi(v.y));
}
__device__ __forceinline__ void rope_store(float* p, F2 a, F2 b) {
  float4 y;
  f2_split(a, y.x, y.y);
  f2_split(b, y.z, y.w);
  *reinterpret_cast<float4*>(p) = y;
}
__device__ __forceinline__ void rope_store(bf16* p, F2 a, F2 b) {
  float4 y;
  f2_split(a, y.x, y.y);
  f2_split(b, y.z, y.w);
  __nv_bfloat162 u = __floats2bfloat162_rn(y.x, y.y), v = __floats2bfloat162_rn(y.z, y.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&u), *reinterpret_cast<uint32_t*>(&v));
}

// What one side's heads are multiplied by for a token: the lane's eight channels
// are x = (x0 x1 | x2 x3) and z, and
//   paired halves:  y = x A + z B,  v = z C + x E        (pair i: x_i with z_i)
//   interleaved:    y = x A + swap(x) B,  v = z C + swap(z) E
struct RopeCoef {
  F2 A[2], B[2], C[2], E[2];
};
template <typename T, bool INTER>
__device__ __forceinline__ RopeCoef rope_coef(const T* w, int c0, int c1, const float (&cs)[4], const float (&sn)[4]) {
  float wx[4], wz[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wx[i] = w ? to_f32(w[c0 + i]) : 1.f;
    wz[i] = w ? to_f32(w[c1 + i]) : 1.f;
  }
  RopeCoef r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (INTER) {
      r.A[i] = f2(wx[2 * i] * cs[i], wx[2 * i + 1] * cs[i]);
      r.B[i] = f2(-wx[2 * i + 1] * sn[i], wx[2 * i] * sn[i]);
      r.C[i] = f2(wz[2 * i] * cs[i + 2], wz[2 * i + 1] * cs[i + 2]);
      r.E[i] = f2(-wz[2 * i + 1] * sn[i + 2], wz[2 * i] * sn[i + 2]);
    } else {
      const int a = 2 * i, b = a + 1;
      r.A[i] = f2(wx[a] * cs[a], wx[b] * cs[b]);
      r.B[i] = f2(-wz[a] * sn[a], -wz[b] * sn[b]);
      r.C[i] = f2(wz[a] * cs[a], wz[b] * cs[b]);
      r.E[i] = f2(wx[a] * sn[a], wx[b] * sn[b]);
    }
  }
  return r;
}
__device__ __forceinline__ F2 f2_swap(F2 v) {
  float a, b;
  f2_split(v, a, b);
  return f2(b, a);
}

// Steps [s0, s1) of one side (queries or keys) of a token: step s holds heads
// s HS .. s HS + HS - 1.  FULL: every channel is rotated.
template <typename T, int D, bool INTER, bool FULL>
__device__ __forceinline__ void rope_side(const T* in, int64_t in_h, T* out, int64_t out_h, const T* w, int heads, int s0,
                                          int s1, int c0, int c1, const float (&cs)[4], const float (&sn)[4], float eps,
                                          int sub, bool rot) {
  constexpr int L = D / 8, HS = 32 / L, U = kRopeUnroll;
  using V = typename Vec4<T>::type;
  const RopeCoef k = rope_coef<T, INTER>(w, c0, c1, cs, sn);
  int h = s0 * HS + sub;
  const int hend = min(heads, s1 * HS);
  in += h * in_h;
  out += h * out_h;
  in_h *= HS;
  out_h *= HS;
  for (int s = s0; s < s1; s += U) {
    V r0[U], r1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r0[u] = r1[u] = V{};
      if (h + u * HS < hend) {
        r0[u] = rope_load(in + c0);
        r1[u] = rope_load(in + c1);
      }
      in += in_h;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u < s1) {
        F2 x[2], z[2];
        rope_unpack(r0[u], x[0], x[1]);
        rope_unpack(r1[u], z[0], z[1]);
        float inv = 1.f;
        if (w) {
          const F2 q = f2_fma(x[0], x[0], f2_fma(x[1], x[1], f2_fma(z[0], z[0], f2_mul(z[1], z[1]))));
          float ss, hi;
          f2_split(q, ss, hi);
          ss += hi;
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          inv = rsqrtf(ss * (1.f / D) + eps);
        }
        const F2 iv = f2(inv, inv);
        F2 y[2], v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // channels that are not rotated do not see their neighbour (0 * inf)
          const F2 xo = INTER ? f2_swap(x[i]) : z[i], zo = INTER ? f2_swap(z[i]) : x[i];
          y[i] = f2_mul(f2_fma(FULL || rot ? xo : 0ull, k.B[i], f2_mul(x[i], k.A[i])), iv);
          v[i] = f2_mul(f2_fma(FULL || rot ? zo : 0ull, k.E[i], f2_mul(z[i], k.C[i])), iv);
        }
        if (h + u * HS < hend) {
          rope_store(out + c0, y[0], y[1]);
          rope_store(out + c1, v[0], v[1]);
        }
      }
      out += out_h;
    }
    h += U * HS;
  }
}

// A warp takes items (a token, or one of its `chunks` shares of `per` steps).
template <typename T, int D, bool INTER, bool FULL>
__global__ void __launch_bounds__(kRopeThreads, kRopePerSm)
qk_norm_rope_kernel(const __grid_constant__ RopeArgs a, int per, int chunks) {
  constexpr int L = D / 8, HS = 32 / L;
  const int lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
  const int half = FULL ? D / 2 : a.R >> 1;
  const bool rot = FULL || 8 * l < a.R;  // R is a multiple of 16: a lane is rotated whole or not at all
  const int c0 = INTER || !rot ? 8 * l : 4 * l, c1 = INTER || !rot ? 8 * l + 4 : half + 4 * l;
  uint64_t f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = rot ? a.freq[4 * l + i] : 0ull;
  const int qsteps = (a.Hq + HS - 1) / HS, steps = qsteps + (a.Hkv + HS - 1) / HS;
  pdl_wait_then_release();
  const int64_t warps = (int64_t)gridDim.x * (kRopeThreads / 32), items = (int64_t)a.N * chunks;
  for (int64_t it = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); it < items; it += warps) {
    const int64_t t = chunks == 1 ? it : it / chunks;
    const int s0 = chunks == 1 ? 0 : (int)(it - t * chunks) * per, s1 = min(s0 + per, steps);
    const int pos = a.pos[t];
    if (pos < 0) continue;
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t turn = (int64_t)((uint64_t)(int64_t)pos * f[i]);
      sincospif((float)turn * 1.0842021724855044e-19f, &sn[i], &cs[i]);  // 2^-63: half turns in [-1, 1]
    }
    if (s0 < qsteps)
      rope_side<T, D, INTER, FULL>(static_cast<const T*>(a.q) + t * a.q_t, a.q_h, static_cast<T*>(a.qo) + t * a.qo_t,
                                   a.qo_h, static_cast<const T*>(a.wq), a.Hq, s0, min(s1, qsteps), c0, c1, cs, sn, a.eps,
                                   sub, rot);
    if (s1 > qsteps)
      rope_side<T, D, INTER, FULL>(static_cast<const T*>(a.k) + t * a.k_t, a.k_h, static_cast<T*>(a.ko) + t * a.ko_t,
                                   a.ko_h, static_cast<const T*>(a.wk), a.Hkv, max(s0 - qsteps, 0), s1 - qsteps, c0, c1,
                                   cs, sn, a.eps, sub, rot);
  }
}

template <typename T, int D, bool INTER>
static cudaError_t rope_launch(const RopeArgs& a, cudaStream_t st) {
  constexpr int HS = 256 / D, NW = kRopeThreads / 32;
  const int steps = (a.Hq + HS - 1) / HS + (a.Hkv + HS - 1) / HS;
  // few tokens: a token's heads go to several warps, up to 8 warps per SM
  const int64_t sms = sm_count();
  const int64_t want = std::min<int64_t>(steps, std::max<int64_t>(1, sms * 8 / a.N));
  const int per = (int)((steps + want - 1) / want), chunks = (steps + per - 1) / per;
  const int64_t ctas = std::min<int64_t>(((int64_t)a.N * chunks + NW - 1) / NW, sms * kRopePerSm);
  const dim3 grid((unsigned)ctas), block(kRopeThreads);
  cudaError_t e = a.R == D ? launch_pdl(qk_norm_rope_kernel<T, D, INTER, true>, grid, block, 0, st, a, per, chunks)
                           : launch_pdl(qk_norm_rope_kernel<T, D, INTER, false>, grid, block, 0, st, a, per, chunks);
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
