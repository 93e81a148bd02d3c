// arith.hpp -- quotients and roots that are rounded once, from the 1-ulp
// instructions and one step of Newton's method: a third of the full division's
// instructions and a third of the root's.  Reciprocal and quotient hold for normal
// arguments and results.  They gave the full ones' bits on all 2^24 mantissas of two octaves.
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
// sqrt(x) of 0 and of x from kRootFrom on: what the correction adds to is an
// exact remainder, 2^-47 of x, and has to be among fp32's numbers.
constexpr float kRootFrom = 0x1p-100f;
__device__ __forceinline__ float root_of(float x) {
  const float r = __builtin_amdgcn_rsqf(__builtin_fmaxf(x, 0x1p-126f)), s = x * r;
  return __builtin_fmaf(__builtin_fmaf(-s, s, x), 0.5f * r, s);
}
// And of all others, by a power of four more.
__device__ __forceinline__ float any_root_of(float x) {
  const bool small = x < kRootFrom;
  return root_of(small ? x * 0x1p64f : x) * (small ? 0x1p-32f : 1.0f);
}

}  // namespace hc
