// adamw_kernels.hip -- an AdamW step over many tensors, states in 32 or 8
// bits, for gfx950.
//
//   g' = c g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// A stream over memory: every value is read and written once, 22 bytes a bf16
// parameter with fp32 states and 10 with states of 8 bits.  The tensors are cut
// into chunks of 2048 values, numbered through all of them, so that one launch
// covers a thousand small vectors and a large matrix evenly.  Their table lies
// in device memory, written once for as long as they stay where they are.  Only
// the lanes that a tensor's end cuts go by single values.
//
// States of 8 bits are e4m3 codes of m and of sqrt(v) with a scale for 128
// values: sqrt halves the orders of magnitude that v spans, so that both fit the
// 17 bits of range that e4m3 has below its block's largest.  A block is 16
// lanes, whose largest magnitude four DPP steps find.  Their step is bound by
// the lanes' work as much as by memory (some 60 instructions a value, the
// random bits' three products, a root and two reciprocals among them), so what is
// stored comes from the 1-ulp instructions with one correction (the parameter's
// own quotient from the reciprocal as it is, 1 ulp), and the conversions round by
// random bits themselves.
//
// Measured in a loop: 2^25 values of 290 views, fp32 states and gradients, mixed
// parameters (808 MB) 150 us, 5.4 TB/s (a large copy: 4.8-5.2); 2^28 bf16 values of
// 450 tensors, 8 bits, random bits (2.72 GB) 536 us, 5.1 TB/s; 3 * 10^5 fp32 values
// of 12 tensors 5.1 us.  By a trace of the kernels, as all variants here are: 149,
// 571 and 5.4; non-temporal loads and stores 162 (2^25 values) and 566 (2^28).
#include <math.h>

#include "arith.hpp"
#include "lanes.hpp"
#include "launch.hpp"
#include "rows.hpp"
#include "step_launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kChunk = 2048;                    // values, 8 a lane
static_assert(kChunk == kThreads * 8, "8 values a lane");
constexpr uint32_t kMostBlocks = 1u << 23;           // of a launch: its lanes are counted in 32 bits
// Chunks in a row for a workgroup.  States of 8 bits are bound by the lanes'
// work, of which looking up a tensor is a part: 2^28 bf16 values of 450 tensors
// take 850 us by 1, 590 by 4, 570 by 8, 566 by 16.  States of 32 bits wait for
// memory, which more workgroups keep busier: 2^25 values, 149 us by 1, 162 by 4.
constexpr uint32_t kRun8 = 8;
constexpr uint32_t kFillBlocks = 2048;               // workgroups that fill the GPU
constexpr uint32_t kPBf16 = 1u << 31, kGBf16 = 1u << 30, kIndex = kGBf16 - 1;
constexpr float kTinyBlock = 0x1p-100f;              // the scale of a block below it would lose its bits

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint16_t* copy;
  uint64_t count;
  float decay;
  uint32_t kind;        // kPBf16, kGBf16 and the tensor's number
};

// An address that was read from memory, known to be one of global memory: else
// its loads are flat ones, which wait for shared memory as well.
template <typename T>
__device__ __forceinline__ T* global(T* p) {
  return (T*)(__attribute__((address_space(1))) T*)(uintptr_t)p;
}

// Chunks begin where the fp32 states are 128-byte aligned (the first begins
// before the tensor), so that stores fill whole lines; blocks of 8-bit states
// count from the tensor's start, and so do their chunks.
__host__ __device__ __forceinline__ uint32_t lead_of(const Tensor& t) {
  return t.ms ? 0 : (uint32_t)((uintptr_t)t.m & 127u) / 4;
}

constexpr uint32_t kPerLaunch = 48;
struct Batch {
  Tensor t[kPerLaunch];
  uint32_t first[kPerLaunch];
};

__global__ void __launch_bounds__(64) adamw_table_kernel(Batch b, uint32_t n, Tensor* t, uint32_t* first) {
  const uint32_t i = threadIdx.x;
  if (i < n) {
    t[i] = b.t[i];
    first[i] = b.first[i];
  }
}

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0xB7E15163u;
  x ^= x >> 15;
  x *= 0x6A09E667u;
  return x ^ (x >> 16);
}
__host__ __device__ __forceinline__ uint32_t step_key(uint64_t seed, int64_t step) {
  return mix(mix(mix((uint32_t)seed) ^ (uint32_t)(seed >> 32)) ^ (uint32_t)step);
}

// The step's numbers as the host has them.
struct Step {
  double beta1, beta2;         // where the device has the step
  float b1, a1, b2, a2;        // a = 1 - b
  float lr, eps, decay;
  float unbias1, unbias2;      // 1 / (1 - b1^t) and 1 / sqrt(1 - b2^t)
  float scale, max_norm;
  const float* d_norm;
  const float* d_lr;
  const int64_t* d_step;
  uint64_t seed;
  uint32_t key;
  int skip;
};

// And as the values use them.
struct Nums {
  float c, b1, a1, b2, a2, rate, unbias2, eps, shrink;   // rate = lr * unbias1, shrink = lr * decay
};

__device__ double power(double b, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1) {
    if (n & 1) r *= b;
    b *= b;
  }
  return r;
}

// False: nothing is to be done.
__device__ __forceinline__ bool numbers(const Step& s, Nums* n, uint32_t* key) {
  n->c = s.scale;
  if (s.d_norm) {
    const float norm = *s.d_norm;
    if (s.skip && !(norm < __builtin_inff())) return false;
    const float q = s.max_norm / (fabsf(s.scale) * norm + 1e-6f);
    n->c = s.scale * (q > 1.0f ? 1.0f : q);       // NaN stays NaN
  }
  const float lr = s.d_lr ? *s.d_lr : s.lr;
  float unbias1 = s.unbias1;
  n->unbias2 = s.unbias2;
  *key = s.key;
  if (s.d_step) {
    const int64_t t = *s.d_step;
    unbias1 = (float)(1.0 / (1.0 - power(s.beta1, t)));
    n->unbias2 = (float)(1.0 / sqrt(1.0 - power(s.beta2, t)));
    *key = step_key(s.seed, t);
  }
  n->b1 = s.b1;
  n->a1 = s.a1;
  n->b2 = s.b2;
  n->a2 = s.a2;
  n->eps = s.eps;
  n->rate = lr * unbias1;
  n->shrink = lr * s.decay;
  return true;
}

// ---------------------------------------------------------------- 8 values of a lane

// Where a lane's 8 values lie: a chunk's first value (the same for all lanes, so
// that addresses are a scalar and an offset), the lane's first one there, and,
// for lanes that a tensor's end cuts, which of the chunk's values exist.
struct Place {
  int64_t at;
  int32_t i, lo, hi;      // lo <= i + j < hi exists
};

// 8 values of an array of T; FULL: all of them exist, else those that do not are
// another value of it and are not stored.
__device__ __forceinline__ int32_t inside(const Place& w, int32_t i) { return i < w.lo ? w.lo : i < w.hi ? i : w.hi - 1; }
template <typename T, bool FULL>
__device__ __forceinline__ void load8(const void* p, const Place& w, vec4* v) {
  const typename T::raw* q = elem<T>(p, 0) + w.at;
  if constexpr (FULL) {
#pragma unroll
    for (int j = 0; j < 8 / T::kVec; ++j) v[j] = load_vec<T>(q + (uint32_t)(w.i + j * T::kVec));
  } else {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = T::widen(q[inside(w, w.i + j)]);
#pragma unroll
    for (int j = 0; j < 8 / T::kVec; ++j) v[j] = T::pack(f + j * T::kVec);
  }
}
template <typename T>
__device__ __forceinline__ void unpack8(const vec4* v, float* f) {
#pragma unroll
  for (int j = 0; j < 8 / T::kVec; ++j) T::unpack(v[j], f + j * T::kVec);
}
template <typename T, bool FULL>
__device__ __forceinline__ void store8(void* p, const Place& w, const float* f) {
  typename T::raw* q = elem<T>(p, 0) + w.at;
  if constexpr (FULL) {
#pragma unroll
    for (int j = 0; j < 8 / T::kVec; ++j) store_vec<T>(q + (uint32_t)(w.i + j * T::kVec), T::pack(f + j * T::kVec));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (w.i + j >= w.lo && w.i + j < w.hi) q[w.i + j] = T::narrow(f[j]);
  }
}

typedef uint32_t codes8 __attribute__((ext_vector_type(2)));
typedef codes8 codes8_u __attribute__((aligned(1)));
template <bool FULL>
__device__ __forceinline__ codes8 load_codes(const void* p, const Place& w) {
  const uint8_t* q = static_cast<const uint8_t*>(p) + w.at;
  if constexpr (FULL) return *reinterpret_cast<const codes8_u*>(q + (uint32_t)w.i);
  codes8 v = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j / 4] |= (uint32_t)q[inside(w, w.i + j)] << (8 * (j % 4));
  return v;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(void* p, const Place& w, codes8 v) {
  uint8_t* q = static_cast<uint8_t*>(p) + w.at;
  if constexpr (FULL) {
    *reinterpret_cast<codes8_u*>(q + (uint32_t)w.i) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (w.i + j < w.hi) q[w.i + j] = (uint8_t)(v[j / 4] >> (8 * (j % 4)));
  }
}
__device__ __forceinline__ void decode8(codes8 v, float* f) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[j], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[j], true);
    f[4 * j] = lo[0];
    f[4 * j + 1] = lo[1];
    f[4 * j + 2] = hi[0];
    f[4 * j + 3] = hi[1];
  }
}
__device__ __forceinline__ codes8 encode8(const float* f) {
  codes8 v;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j], f[4 * j + 1], 0, false);
    v[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j + 2], f[4 * j + 3], w, true);
  }
  return v;
}

// Eight values of each of 16 lanes, as codes and the block's scale.  A NaN or an
// infinity makes the scale one, and with it the block.
// The instruction that rounds by random bits adds the 32 it is given to what a
// code cuts off, aligned at the top: here 16 of them and a half.
template <bool SEEDED, bool ROOT>
__device__ __forceinline__ codes8 quantise(const float* x, const uint32_t* bits, float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, ROOT ? f32_bits(x[j]) : f32_bits(x[j]) & 0x7FFFFFFFu);
  const float a = bits_f32(join_lanes<16>(top, MaxOp{}));
  const bool tiny = a < kTinyBlock;
  const float unit = a * (1.0f / 448.0f), inv = tiny ? 0.0f : reciprocal(unit);
  *scale = tiny ? 0.0f : unit;
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float least = ROOT ? (x[j] > 0.0f ? 0x1p-9f : 0.0f) : -448.0f;
    y[j] = __builtin_amdgcn_fmed3f(quotient(x[j], unit, inv), least, 448.0f);
  }
  if constexpr (!SEEDED) return encode8(y);
  codes8 v = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = ROOT ? (bits[4 * j + i] & 0xFFFF0000u) | 0x8000u : bits[4 * j + i] << 16 | 0x8000u;
    int w = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * j], (int)r[0], 0, 0);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * j + 1], (int)r[1], w, 1);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * j + 2], (int)r[2], w, 2);
    v[j] = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(y[4 * j + 3], (int)r[3], w, 3);
  }
  return v;
}

// ---------------------------------------------------------------- chunks

template <typename P, typename G, int BITS, bool SEEDED, bool FULL>
__device__ __forceinline__ void lane_body(const Tensor& t, const Place& w, const Nums& n, uint32_t key) {
  const float decay = n.shrink * t.decay;
  const uint32_t key0 = mix(key ^ (uint32_t)((uint64_t)w.at >> 32));
  const uint32_t key1 = mix(key ^ (uint32_t)((uint64_t)(w.at + kChunk - 1) >> 32));
  vec4 p[8 / P::kVec], g[8 / G::kVec], m[2], v[2];
  codes8 mc, vc;
  float ms, vs;
  load8<P, FULL>(t.p, w, p);
  load8<G, FULL>(t.g, w, g);
  if constexpr (BITS == 32) {
    load8<F32, FULL>(t.m, w, m);
    load8<F32, FULL>(t.v, w, v);
  } else {
    mc = load_codes<FULL>(t.m, w);
    vc = load_codes<FULL>(t.v, w);
    // a chunk begins with a block, and a lane that its block keeps here may lie past the end, within it
    ms = (t.ms + w.at / HC_STATE_BLOCK)[(uint32_t)w.i / HC_STATE_BLOCK];
    vs = (t.vs + w.at / HC_STATE_BLOCK)[(uint32_t)w.i / HC_STATE_BLOCK];
  }
  float fp[8], fg[8], fm[8], fv[8], root[8];
  unpack8<P>(p, fp);
  unpack8<G>(g, fg);
  if constexpr (BITS == 32) {
    unpack8<F32>(m, fm);
    unpack8<F32>(v, fv);
  } else {
    decode8(mc, fm);
    decode8(vc, fv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      fm[j] *= ms;
      fv[j] *= vs;
      fv[j] *= fv[j];
    }
  }
  uint32_t least = ~0u;      // v that is not 0, and how it lies: v is not negative
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = fg[j] * n.c;
    fm[j] = n.b1 * fm[j] + n.a1 * x;
    fv[j] = n.b2 * fv[j] + n.a2 * (x * x);
    root[j] = BITS == 8 ? root_of(fv[j]) : __builtin_sqrtf(fv[j]);
    if (BITS == 8) least = min(least, f32_bits(fv[j]) - 1);
  }
  if (BITS == 8 && least < f32_bits(kRootFrom) - 1) {      // few lanes: 536 us of 2^28 values with and without
#pragma unroll
    for (int j = 0; j < 8; ++j) root[j] = any_root_of(fv[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float den = __builtin_fmaf(root[j], n.unbias2, n.eps);
    fp[j] = __builtin_fmaf(-decay, fp[j], fp[j]);
    fp[j] = BITS == 8 ? __builtin_fmaf(-n.rate * fm[j], __builtin_amdgcn_rcpf(den), fp[j])
                      : fp[j] - n.rate * fm[j] / den;
  }
  uint32_t bits[8];
  if constexpr (SEEDED) {
    // blocks of 8 bits, and so lanes, begin at multiples of 8; a chunk of the
    // others may reach over a multiple of 2^32
    const uint32_t from = (uint32_t)w.at * 0x9E3779B9u + (uint32_t)w.i * 0x9E3779B9u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool over = BITS == 32 && (uint32_t)w.at + (uint32_t)(w.i + j) < (uint32_t)w.at;
      bits[j] = mix((over ? key1 : key0) + (from + (uint32_t)j * 0x9E3779B9u));
    }
  }
  if constexpr (SEEDED && P::kVec == 8) {
    if constexpr (FULL) {
      vec4 o4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        b2 o = {};
        o = __builtin_amdgcn_cvt_sr_bf16_f32(o, fp[2 * j], bits[2 * j] * 0x9E3779B9u, false);
        o = __builtin_amdgcn_cvt_sr_bf16_f32(o, fp[2 * j + 1], bits[2 * j + 1] * 0x9E3779B9u, true);
        o4[j] = __builtin_bit_cast(uint32_t, o);
      }
      store_vec<P>(elem<P>(t.p, 0) + w.at + (uint32_t)w.i, o4);
    } else {
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t x = (f32_bits(fp[j]) + ((bits[j] * 0x9E3779B9u) >> 16)) & 0xFFFF0000u;
        r[j] = fp[j] == fp[j] ? bits_f32(x) : fp[j];
      }
      store8<P, FULL>(t.p, w, r);
    }
  } else {
    store8<P, FULL>(t.p, w, fp);
    if constexpr (P::kVec == 4)
      if (t.copy) store8<BF16, FULL>(t.copy, w, fp);
  }
  if constexpr (BITS == 32) {
    store8<F32, FULL>(t.m, w, fm);
    store8<F32, FULL>(t.v, w, fv);
  } else {
    if constexpr (!FULL) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (w.i + j >= w.hi) fm[j] = root[j] = 0.0f;      // no part of the block's largest
    }
    float sm, sv;
    const codes8 qm = quantise<SEEDED, false>(fm, bits, &sm), qv = quantise<SEEDED, true>(root, bits, &sv);
    store_codes<FULL>(t.m, w, qm);
    store_codes<FULL>(t.v, w, qv);
    if ((uint32_t)w.i % HC_STATE_BLOCK == 0) {
      (t.ms + w.at / HC_STATE_BLOCK)[(uint32_t)w.i / HC_STATE_BLOCK] = sm;
      (t.vs + w.at / HC_STATE_BLOCK)[(uint32_t)w.i / HC_STATE_BLOCK] = sv;
    }
  }
}

// The lanes of a chunk, those that a tensor's end cuts by single values: with
// 8 bits all 16 of its block, since a block's largest is found among them.
template <typename P, typename G, int BITS, bool SEEDED>
__device__ __forceinline__ void chunk_of(const Tensor& t, int64_t at, const Nums& n, uint32_t key) {
  const int64_t left = (int64_t)t.count - at;
  const int32_t i = (int32_t)threadIdx.x * 8;
  const Place w = {at, i, at < 0 ? (int32_t)-at : 0, left < kChunk ? (int32_t)left : (int32_t)kChunk};
  const int32_t first = BITS == 32 ? i : i - i % HC_STATE_BLOCK, end = first + (BITS == 32 ? 8 : HC_STATE_BLOCK);
  if (first >= w.lo && end <= w.hi)
    lane_body<P, G, BITS, SEEDED, true>(t, w, n, key);
  else if (first < w.hi && end > w.lo)
    lane_body<P, G, BITS, SEEDED, false>(t, w, n, key);
}

// A workgroup takes `run` chunks in a row: a tensor is looked up once for those
// that it has of them.
template <int BITS, bool SEEDED>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const Tensor* tensors, const uint32_t* first, uint32_t n,
                                                         uint32_t chunks, uint32_t run, Step s) {
  Nums nums;
  uint32_t key;
  if (!numbers(s, &nums, &key)) return;
  uint32_t c = blockIdx.x * run;
  const uint32_t end = min(chunks, c + run);
  while (c < end) {
    const uint32_t k = find_tensor(first, n, c);
    Tensor t = tensors[k];
    t.p = global(t.p);
    t.g = global(t.g);
    t.m = global(t.m);
    t.v = global(t.v);
    t.ms = global(t.ms);
    t.vs = global(t.vs);
    t.copy = global(t.copy);
    const uint32_t own = SEEDED ? mix(key ^ (t.kind & kIndex)) : 0;
    const uint32_t last = k + 1 < n ? min(end, first[k + 1]) : end;
    const int64_t at = (int64_t)(c - first[k]) * kChunk - lead_of(t);
    auto go = [&](auto p, auto g) {
      int64_t x = at;
      for (uint32_t i = c; i < last; ++i, x += kChunk) chunk_of<decltype(p), decltype(g), BITS, SEEDED>(t, x, nums, own);
    };
    if (t.kind & kPBf16) {
      if (t.kind & kGBf16)
        go(BF16{}, BF16{});
      else
        go(BF16{}, F32{});
    } else {
      if (t.kind & kGBf16)
        go(F32{}, BF16{});
      else
        go(F32{}, F32{});
    }
    c = last;
  }
}

}  // namespace

size_t adamw_table_bytes(size_t n) { return (n * (sizeof(Tensor) + sizeof(uint32_t)) + 15) & ~(size_t)15; }

hipError_t launch_adamw_plan(hc_adamw_plan_t* plan, const AdamWTensor* tensors, size_t n, void* table,
                             hipStream_t stream) {
  Tensor* t = static_cast<Tensor*>(table);
  uint32_t* firsts = reinterpret_cast<uint32_t*>(t + n);
  uint64_t chunks = 0;
  Batch b;
  uint32_t k = 0;
  size_t done = 0;
  for (size_t i = 0; i < n; ++i) {
    const AdamWTensor& x = tensors[i];
    b.t[k] = Tensor{x.p, x.g, x.m, x.v, x.ms, x.vs, static_cast<uint16_t*>(x.copy), x.count, x.decay,
                    (uint32_t)x.index | (x.p_dtype == HC_BF16 ? kPBf16 : 0) | (x.g_dtype == HC_BF16 ? kGBf16 : 0)};
    b.first[k] = (uint32_t)chunks;
    chunks += (x.count + lead_of(b.t[k]) + kChunk - 1) / kChunk;
    if (chunks > 0x7FFFFFFFull) return hipErrorInvalidValue;     // 2^42 values
    ++k;
    if (k == kPerLaunch || done + k == n) {
      HC_ENQUEUE(adamw_table_kernel, 1, 64, stream, b, k, t + done, firsts + done);
      done += k;
      k = 0;
    }
  }
  plan->ntensors = n;
  plan->chunks = chunks;
  plan->d_table = table;
  return hipSuccess;
}

hipError_t launch_adamw(const hc_adamw_plan_t& plan, const hc_adamw_opts_t& o, hipStream_t stream) {
  if (!plan.chunks) return hipSuccess;
  const double t = (double)(o.step > 0 ? o.step : 1);
  Step s = {};
  s.beta1 = o.beta1;
  s.beta2 = o.beta2;
  s.b1 = (float)o.beta1;
  s.a1 = (float)(1.0 - o.beta1);
  s.b2 = (float)o.beta2;
  s.a2 = (float)(1.0 - o.beta2);
  s.lr = (float)o.lr;
  s.eps = (float)o.eps;
  s.decay = (float)o.weight_decay;
  s.unbias1 = (float)(1.0 / (1.0 - pow(o.beta1, t)));
  s.unbias2 = (float)(1.0 / sqrt(1.0 - pow(o.beta2, t)));
  s.scale = o.grad_scale;
  s.max_norm = o.max_norm;
  s.d_norm = o.d_norm;
  s.d_lr = o.d_lr;
  s.d_step = o.d_step;
  s.seed = o.seed;
  s.key = step_key(o.seed, o.step);
  s.skip = o.skip_nonfinite;
  const Tensor* table = static_cast<const Tensor*>(plan.d_table);
  const uint32_t* firsts = reinterpret_cast<const uint32_t*>(table + plan.ntensors);
  const uint32_t n = (uint32_t)plan.ntensors, chunks = (uint32_t)plan.chunks;
  uint32_t run = 1;
  if (plan.state_bits == 8)
    while (run < kRun8 && chunks / run >= 2 * kFillBlocks) run *= 2;
  while (chunks / run >= kMostBlocks) run *= 2;
  const uint32_t grid = (uint32_t)(((uint64_t)chunks + run - 1) / run);
  auto launch = [&](auto kernel) {
    HC_ENQUEUE(kernel, grid, kThreads, stream, table, firsts, n, chunks, run, s);
    return hipSuccess;
  };
  if (plan.state_bits == 32) return o.seed ? launch(adamw_kernel<32, true>) : launch(adamw_kernel<32, false>);
  return o.seed ? launch(adamw_kernel<8, true>) : launch(adamw_kernel<8, false>);
}

}  // namespace hc
