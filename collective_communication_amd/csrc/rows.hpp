// rows.hpp -- device helpers of the kernels that move and sum rows of fp32 or
// bf16 elements (gradients, embedding rows, tokens of experts).
//
// Accesses are 16-byte vectors that are only element aligned (a gradient that
// is added to its table reads and writes the table by elements): gfx950 runs in
// unaligned access mode, so a row that starts at an odd element (an odd
// width, a bucket's view) takes the same wide path as an aligned one.  A
// row's last vector is moved back to end where the row ends (vec_at): the
// elements that it shares with the vector before it are read twice, computed
// alike and written twice with the same values, and no lane branches.  Rows
// narrower than one vector go by single elements (the types ending in S).
// Measured, combine of 4068 tokens x 6 slots x 1031 bf16: 11.7 us so, 18.6
// with the last vector's elements taken one by one; 1024 x 6 x 4095, 10.9 and
// 17.7, against 10.4 at a width of 4096.
// Values are widened to fp32 exactly and rounded once (nearest even) where
// they are stored as bf16.
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
// The experts' calls count a row for every slot, since the host does not know
// which are another rank's: one of eight ranks stores 16 MB of rows so and loads
// 32 MB so.  8000 tokens x 8 slots x 4096 bf16 there (66 MB of rows), counted
// by slots / by own rows, us: dispatch 17.8 / 22.3, and a copy of its rows
// behind it 45.3 / 40.8; combine 24.9 / 20.6, its input just written 23.7 / 22.7;
// its gradient 30.3 / 32.0, and a copy behind it 54.6 / 51.4.  2000 tokens: the
// same within 3%.
constexpr size_t kStreamStoreBytes = (size_t)128 << 20;

// And launches that read at least this many bytes of rows, each once, load
// them non-temporal: what comes straight from its producer is mostly in the
// 256 MB Infinity Cache below that, and from memory above.  The combine of rows
// of 4096 bf16, plain / non-temporal, us, its input just written: 134 MB 23 /
// 26, 268 MB 48 / 53, 393 MB 87 / 76, 1.07 GB 224 / 210; three inputs in turn
// (nothing cached): 134 MB 32 / 28, 268 MB 61 / 54, 393 MB 88 / 77.
constexpr size_t kStreamLoadBytes = (size_t)256 << 20;

typedef uint32_t vec4 __attribute__((ext_vector_type(4)));
typedef vec4 vec4_u __attribute__((aligned(2)));   // element aligned

// Element type tags: kVec elements are what a lane moves at once, a T::vec.
struct F32 {
  typedef uint32_t raw;
  typedef vec4 vec;
  static constexpr int kVec = 4;
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
  typedef vec4 vec;
  static constexpr int kVec = 8;
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

// One element per lane.
template <typename T>
struct Single {
  typedef typename T::raw raw;
  typedef typename T::raw vec;
  static constexpr int kVec = 1;
  static __device__ __forceinline__ void unpack(vec v, float* f) { f[0] = T::widen(v); }
  static __device__ __forceinline__ vec pack(const float* f) { return T::narrow(f[0]); }
  static __device__ __forceinline__ float widen(raw x) { return T::widen(x); }
  static __device__ __forceinline__ raw narrow(float f) { return T::narrow(f); }
};
typedef Single<F32> F32S;
typedef Single<BF16> BF16S;

template <typename T>
__device__ __forceinline__ const typename T::raw* elem(const void* p, size_t i) {
  return static_cast<const typename T::raw*>(p) + i;
}
template <typename T>
__device__ __forceinline__ typename T::raw* elem(void* p, size_t i) {
  return static_cast<typename T::raw*>(p) + i;
}

// Where the vector that begins at column c is read and written: there, or,
// for the last one of a row of dim >= kVec, so that it ends with the row.
template <typename T>
__device__ __forceinline__ uint32_t vec_at(uint32_t c, uint32_t dim) {
  return c + T::kVec <= dim ? c : dim - T::kVec;
}

template <typename T, bool NT = false>
__device__ __forceinline__ typename T::vec load_vec(const typename T::raw* p) {
  if constexpr (T::kVec == 1) {
    return NT ? __builtin_nontemporal_load(p) : *p;
  } else {
    const vec4_u* q = reinterpret_cast<const vec4_u*>(p);
    return NT ? __builtin_nontemporal_load(q) : *q;
  }
}
template <typename T, bool NT = false>
__device__ __forceinline__ void store_vec(typename T::raw* p, typename T::vec v) {
  if constexpr (T::kVec == 1) {
    if constexpr (NT)
      __builtin_nontemporal_store(v, p);
    else
      *p = v;
  } else {
    vec4_u* q = reinterpret_cast<vec4_u*>(p);
    if constexpr (NT)
      __builtin_nontemporal_store((vec4_u)v, q);
    else
      *q = v;
  }
}
template <typename T>
__device__ __forceinline__ typename T::vec zero_vec() {
  if constexpr (T::kVec == 1)
    return 0;
  else
    return vec4{0, 0, 0, 0};
}

// The N (1, 4 or 8) fp32 values of a lane as N elements of To (F32 or BF16).
template <typename To, int N>
__device__ __forceinline__ void store_vals(typename To::raw* p, const float* f) {
  if constexpr (N == 1) {
    *p = To::narrow(f[0]);
  } else if constexpr (N < To::kVec) {
    typedef uint32_t vec2_u __attribute__((ext_vector_type(2), aligned(2)));
    *reinterpret_cast<vec2_u*>(p) = vec2_u{BF16::pair(f[0], f[1]), BF16::pair(f[2], f[3])};
  } else {
#pragma unroll
    for (int i = 0; i < N; i += To::kVec) store_vec<To>(p + i, To::pack(f + i));
  }
}

// A span of zeroes, `bytes` (a multiple of 2) from p on, by `lanes` lanes;
// NT: stored non-temporal.
template <bool NT>
__device__ __forceinline__ void zero_span(char* p, uint64_t bytes, uint32_t lane, uint32_t lanes) {
  if (bytes < 16) {
    if (lane < bytes / 2) reinterpret_cast<uint16_t*>(p)[lane] = 0;
    return;
  }
  for (uint64_t i = lane * 16; i < bytes; i += lanes * 16)
    store_vec<F32, NT>(reinterpret_cast<uint32_t*>(p + (i + 16 <= bytes ? i : bytes - 16)), vec4{0, 0, 0, 0});
}

__device__ __forceinline__ uint32_t lane_id() { return threadIdx.x & 63u; }
// The wave's number in its workgroup, as a scalar.
__device__ __forceinline__ uint32_t wave_id() { return first_lane_read(threadIdx.x >> 6); }

// The tensor that holds chunk c, the last whose first chunk is not after it:
// a search over 64 places at a time, one per lane, so two loads in turn find
// it among 4096 tensors.  Every lane of the wave calls it.
__device__ __forceinline__ uint32_t find_tensor(const uint32_t* first, uint32_t n, uint32_t c) {
  uint32_t lo = 0;
  while (n > 1) {
    const uint32_t step = (n + 63) / 64, at = lane_id() * step;
    const uint64_t not_after = __ballot(at < n && first[lo + at] <= c);
    const uint32_t skip = ((uint32_t)__popcll(not_after) - 1) * step;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return first_lane_read(lo);
}

}  // namespace hc
