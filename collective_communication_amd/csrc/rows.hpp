// rows.hpp -- device helpers of the kernels that move and sum rows of fp32 or
// bf16 elements (gradients, embedding rows, tokens of experts).
//
// Every access is a 16-byte vector that is only element aligned: gfx950 runs
// in unaligned access mode, so a row that starts at an odd element (an odd
// width, a bucket's view) takes the same wide path as an aligned one.  A
// row's last, partial vector goes element by element.  Values are widened to
// fp32 exactly and rounded once (nearest even) where they are stored as bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "hc.h"

namespace hc {

// Launches whose output has at least this many bytes store it non-temporal.
// Such a store is faster by itself (a lookup of 30,011 x 4096 bf16: 59 us
// plain, 41 us non-temporal), but the next reader finds less of it in the
// caches.  Lookup and a copy of its output together, plain / non-temporal, us:
// 67 MB 42 / 46, 134 MB 96 / 94, 201 MB 151 / 149, 537 MB 388 / 373.
constexpr size_t kStreamStoreBytes = (size_t)128 << 20;

typedef uint32_t vec4 __attribute__((ext_vector_type(4)));
typedef vec4 vec4_u __attribute__((aligned(2)));   // element aligned

// Element type tags: kVec elements fill a 16-byte vector.
struct F32 {
  typedef uint32_t raw;
  static constexpr int kVec = 4;
  static constexpr hc_dtype_t kDtype = HC_F32;
  static __device__ __forceinline__ void unpack(vec4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = bits_f32(v[i]);
  }
  static __device__ __forceinline__ vec4 pack(const float* f) {
    vec4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f32_bits(f[i]);
    return v;
  }
  static __device__ __forceinline__ float widen(raw x) { return bits_f32(x); }
  static __device__ __forceinline__ raw narrow(float f) { return f32_bits(f); }
};

struct BF16 {
  typedef uint16_t raw;
  static constexpr int kVec = 8;
  static constexpr hc_dtype_t kDtype = HC_BF16;
  static __device__ __forceinline__ void unpack(vec4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bits_f32(v[i] << 16);
      f[2 * i + 1] = bits_f32(v[i] & 0xFFFF0000u);
    }
  }
  // The conversion instruction rounds to nearest even and keeps NaN a NaN.
  static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const f2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
  }
  static __device__ __forceinline__ vec4 pack(const float* f) {
    vec4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
    return v;
  }
  static __device__ __forceinline__ float widen(raw x) { return bits_f32((uint32_t)x << 16); }
  static __device__ __forceinline__ raw narrow(float f) { return (raw)pair(f, 0.0f); }
};

template <typename T>
__device__ __forceinline__ const typename T::raw* elem(const void* p, size_t i) {
  return static_cast<const typename T::raw*>(p) + i;
}
template <typename T>
__device__ __forceinline__ typename T::raw* elem(void* p, size_t i) {
  return static_cast<typename T::raw*>(p) + i;
}

// The vector at element p of a row with `left` (>= 1) elements from p on;
// elements past the row's end read as zero and are not touched.
template <typename T, bool NT = false>
__device__ __forceinline__ vec4 load_vec(const typename T::raw* p, uint32_t left) {
  if (left >= T::kVec) {
    if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const vec4_u*>(p));
    return *reinterpret_cast<const vec4_u*>(p);
  }
  vec4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < T::kVec; ++i)
    if ((uint32_t)i < left) {
      if constexpr (T::kVec == 4)
        v[i] = p[i];
      else
        v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  return v;
}

template <typename T, bool NT = false>
__device__ __forceinline__ void store_vec(typename T::raw* p, vec4 v, uint32_t left) {
  if (left >= T::kVec) {
    if constexpr (NT)
      __builtin_nontemporal_store((vec4_u)v, reinterpret_cast<vec4_u*>(p));
    else
      *reinterpret_cast<vec4_u*>(p) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < T::kVec; ++i)
    if ((uint32_t)i < left) {
      if constexpr (T::kVec == 4)
        p[i] = v[i];
      else
        p[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
}

// Stores kVec fp32 values of one lane as elements of type To; for a bf16
// input with an fp32 output that is two vectors.
template <typename To, int N, bool NT = false>
__device__ __forceinline__ void store_vals(typename To::raw* p, const float* f, uint32_t left) {
#pragma unroll
  for (int i = 0; i < N; i += To::kVec) {
    if constexpr (N < To::kVec) {
      // fp32 lanes (4 values) into bf16: half a vector
#pragma unroll
      for (int j = 0; j < N; ++j)
        if ((uint32_t)j < left) p[j] = To::narrow(f[j]);
    } else {
      if ((uint32_t)i < left) store_vec<To, NT>(p + i, To::pack(f + i), left - i);
    }
  }
}
template <typename Ti, int N>
__device__ __forceinline__ void load_vals(const typename Ti::raw* p, float* f, uint32_t left) {
  if constexpr (N < Ti::kVec) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = (uint32_t)j < left ? Ti::widen(p[j]) : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += Ti::kVec) {
      const vec4 v = (uint32_t)i < left ? load_vec<Ti>(p + i, left - i) : vec4{0, 0, 0, 0};
      Ti::unpack(v, f + i);
    }
  }
}

__device__ __forceinline__ uint32_t lane_id() { return threadIdx.x & 63u; }
// The wave's number in its workgroup, as a scalar.
__device__ __forceinline__ uint32_t wave_id() { return first_lane_read(threadIdx.x >> 6); }

}  // namespace hc
