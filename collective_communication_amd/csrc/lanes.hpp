// lanes.hpp -- values joined over neighbouring lanes of a wave, by DPP within 16
// lanes and by swapping halves beyond, with no shared memory.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace hc {

// x of the lane that a step pairs: step 1 lane ^ 1, 2 lane ^ 2, 4 the mirrored
// lane of 8, 8 of 16, which serve where lanes of 4 and 8 already agree.
template <uint32_t STEP>
__device__ __forceinline__ uint32_t lane_pair(uint32_t x) {
  constexpr int ctrl = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, 0xF, 0xF, true);
}

// One step of a join: the 2 * STEP lanes that hold v in two halves, each its own.
template <uint32_t STEP, typename Op>
__device__ __forceinline__ uint32_t join_step(uint32_t v, Op op) {
  if constexpr (STEP < 16) {
    return op(v, lane_pair<STEP>(v));
  } else if constexpr (STEP == 16) {
    const auto x = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return op((uint32_t)x[0], (uint32_t)x[1]);
  } else {
    const auto x = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return op((uint32_t)x[0], (uint32_t)x[1]);
  }
}

// v joined over each LANES (a power of two, at most 64) neighbouring lanes, in all
// of them.
template <uint32_t LANES, typename Op>
__device__ __forceinline__ uint32_t join_lanes(uint32_t v, Op op) {
  if constexpr (LANES > 1) v = join_step<1>(v, op);
  if constexpr (LANES > 2) v = join_step<2>(v, op);
  if constexpr (LANES > 4) v = join_step<4>(v, op);
  if constexpr (LANES > 8) v = join_step<8>(v, op);
  if constexpr (LANES > 16) v = join_step<16>(v, op);
  if constexpr (LANES > 32) v = join_step<32>(v, op);
  return v;
}
template <uint32_t LANES, typename Op>
__device__ __forceinline__ float join_lanes(float v, Op op) {
  return bits_f32(join_lanes<LANES>(f32_bits(v), [&](uint32_t a, uint32_t b) {
    return f32_bits(op(bits_f32(a), bits_f32(b)));
  }));
}

struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// The larger; of a NaN and a number either may come.
struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a > b ? a : b; }
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

}  // namespace hc
