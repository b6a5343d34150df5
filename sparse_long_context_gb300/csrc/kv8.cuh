// The 8-bit cache's code formats: a code c stands for c * s with its block's
// scale s (int8: s = amax / 127; e4m3: s = amax / 448).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace sls {

constexpr int kKv8Int8 = 0, kKv8E4m3 = 1;

template <int FMT> __device__ __forceinline__ float kv8_top() { return FMT == kKv8Int8 ? 127.f : 448.f; }

// The code of x in a block whose largest magnitude is amax (> 0, finite).
// x * top is exact for bf16 x (at most 8 + 7 significant bits), so the
// quotient is rounded once and lies on a tie between two codes only when the
// exact quotient does: the code is that of exact arithmetic.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_code(float x, float amax) {
  const float y = __fdiv_rn(x * kv8_top<FMT>(), amax);
  if constexpr (FMT == kKv8Int8) return (uint32_t)__float2int_rn(y) & 0xffu;
  return __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
}

}  // namespace sls
