// Ranking keys of page scores, with the pages whose scores are not numbers.
//
// A page's score is the largest of its heads' bounds U = sum_c max(q_c kmin_c, q_c kmax_c), which the scorers form as
// kmax . max(q, 0) + kmin . min(q, 0).  The two are the same while the summaries are finite; an infinite side
// that a bound does not take meets a zero there, and 0 inf is NaN.  So pages with a NaN sum are scored anew, by a
// warp each, channel by channel by the side that the query's sign takes; a query that is zero or NaN adds nothing.  What
// is NaN then (infinities of both signs, a NaN summary) could be any number: the page ranks above every score and
// below the forced pages.
#pragma once

#include "common.cuh"

namespace sls {

constexpr uint32_t kNoScoreKey = 0xfffffffeu;  // above the key of +inf, below a forced page's

// The larger value; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The key of a score: kNoScoreKey where it is NaN.
__device__ __forceinline__ uint32_t score_key(float f) { return f != f ? kNoScoreKey : float_key(f); }

// The key of a page from its definition: q [G, D], summaries lo and hi [D] (null: zeros), D 64 or 128.  A warp calls it for one
// page: a lane takes every 32nd channel.
template <typename T>
__device__ __noinline__ uint32_t defined_page_key(const T* q, const T* lo, const T* hi, int G, int D) {
  constexpr int N = 4;
  const int lane = threadIdx.x & 31;
  float l[N], h[N], best = kNegInf;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = lane + 32 * i;
    l[i] = lo && c < D ? to_f32(lo[c]) : 0.f;
    h[i] = lo && c < D ? to_f32(hi[c]) : 0.f;
  }
#pragma unroll 1
  for (int g = 0; g < G; ++g, q += D) {
    float x[N], s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lane + 32 * i < D ? to_f32(q[lane + 32 * i]) : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (x[i] > 0.f) s = fmaf(x[i], h[i], s);
      else if (x[i] < 0.f) s = fmaf(x[i], l[i], s);
    }
    best = max_nan(best, warp_sum(s));
  }
  return score_key(best);
}

}  // namespace sls
