// Per-head root-mean-square norm of queries and keys and the rotation by the
// token's position in one pass over the projected heads:
//   y = x w / sqrt(mean(x^2) + eps),  (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin).
// Bound by memory (every element read and written once).  A head is D/V lanes
// of one 16-byte vector each (V channels), so a warp takes 32 V / D heads at a
// time; a lane keeps the cosines and sines of its own channels for all heads of
// the token, and a half-split pair's other channel is one shuffle away.
//
// Angles are kept in turns: positions[t] * f_i modulo one turn is the low 64
// bits of the product with the frequency as a 64-bit fixed-point fraction
// (one turn = 2^64), exact for every position, so only the frequency's own
// rounding (2^-56 turns) is multiplied by the position.
#include "common.cuh"
#include "launch.h"

namespace sls {

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(256)
qk_norm_rope_kernel(const __grid_constant__ RopeArgs a, int heads_per_warp, int chunks) {
  constexpr int V = Vec16<T>::N;  // channels of a lane
  constexpr int L = D / V;        // lanes of a head
  constexpr int HS = 32 / L;      // heads of one warp step
  constexpr int NA = INTER ? V / 2 : V;
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (item >= (int64_t)a.N * chunks) return;
  const int t = (int)(item / chunks), hc = (int)(item % chunks);
  const int pos = a.pos[t];
  if (pos < 0) return;
  const int sub = lane / L, c0 = (lane % L) * V;
  const int H = a.Hq + a.Hkv, half = a.R >> 1;
  const bool rot = c0 < a.R;  // R is a multiple of 16: a lane is rotated whole or not at all
  float cs[NA], sn[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int f = INTER ? (c0 >> 1) + i : (c0 + i < half ? c0 + i : c0 + i - half);
    const uint64_t turn = (uint64_t)(int64_t)pos * (rot ? a.freq[f] : 0ull);
    const float x = (float)(int64_t)turn * 1.0842021724855044e-19f;  // 2^-63: half turns in [-1, 1]
    sincospif(x, &sn[i], &cs[i]);
    if (!INTER && c0 < half) sn[i] = -sn[i];
  }
  // half-split: the lane holding the pair's other channels
  const int partner = !rot ? lane : (c0 < half ? lane + half / V : lane - half / V);
  float wq[V], wk[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    wq[i] = a.wq ? to_f32(static_cast<const T*>(a.wq)[c0 + i]) : 1.f;
    wk[i] = a.wk ? to_f32(static_cast<const T*>(a.wk)[c0 + i]) : 1.f;
  }
  const int h0 = hc * heads_per_warp, h1 = min(h0 + heads_per_warp, H);
  for (int hs = h0; hs < h1; hs += HS) {
    const int h = hs + sub;
    const bool live = h < h1, isq = h < a.Hq;
    const T* src = isq ? static_cast<const T*>(a.q) + t * a.q_t + h * a.q_h
                       : static_cast<const T*>(a.k) + t * a.k_t + (int64_t)(h - a.Hq) * a.k_h;
    T* dst = isq ? static_cast<T*>(a.qo) + t * a.qo_t + h * a.qo_h
                 : static_cast<T*>(a.ko) + t * a.ko_t + (int64_t)(h - a.Hq) * a.ko_h;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (live) raw = *reinterpret_cast<const uint4*>(src + c0);
    float x[V];
    unpack_vec(raw, x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (isq ? a.wq != nullptr : a.wk != nullptr) {
      const float inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = x[i] * inv * (isq ? wq[i] : wk[i]);
    }
    float y[V];
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        y[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
        y[2 * i + 1] = x[2 * i + 1] * cs[i] + x[2 * i] * sn[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float other = __shfl_sync(0xffffffffu, x[i], partner);
        y[i] = fmaf(other, sn[i], x[i] * cs[i]);
      }
    }
    if (!rot) {
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = x[i];
    }
    if (live) {
      alignas(16) T out[V];
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = from_f32<T>(y[i]);
      *reinterpret_cast<uint4*>(dst + c0) = *reinterpret_cast<const uint4*>(out);
    }
  }
}

template <typename T, int D, bool INTER>
static cudaError_t rope_launch(const RopeArgs& a, cudaStream_t st) {
  constexpr int HS = 32 / (D / Vec16<T>::N);
  const int H = a.Hq + a.Hkv, steps = (H + HS - 1) / HS;
  // few tokens: a token's heads are spread over several warps, until the GPU has about 8 warps per SM
  const int64_t want = ((int64_t)sm_count() * 8 + a.N - 1) / a.N;
  const int per = (int)((steps + (want < steps ? want : steps) - 1) / (want < steps ? want : steps));
  const int chunks = (steps + per - 1) / per;
  const int64_t warps = (int64_t)a.N * chunks;
  const int nw = 4;
  cudaError_t e = launch_pdl(qk_norm_rope_kernel<T, D, INTER>, dim3((unsigned)((warps + nw - 1) / nw)), dim3(nw * 32),
                             0, st, a, per * HS, chunks);
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
