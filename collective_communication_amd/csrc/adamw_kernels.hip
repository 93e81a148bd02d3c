// adamw_kernels.hip -- an AdamW step over many tensors, states in 32 or 8
// bits, for gfx950.
//
//   g' = c g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// A stream over memory: every value is read and written once, 22 bytes a bf16
// parameter with fp32 states and 10 with states of 8 bits.  The tensors are cut
// into chunks of 4096 values, numbered through all of them, so that one launch
// covers a thousand small vectors and a large matrix evenly.  Their table lies
// in device memory, written once for as long as they stay where they are.
//
// States of 8 bits are e4m3 codes of m and of sqrt(v) with a scale for 128
// values: sqrt halves the orders of magnitude that v spans, so that both fit the
// 17 bits of range that e4m3 has below its block's largest.  A block is 16
// lanes, whose largest magnitude four DPP steps find.
#include <math.h>

#include "launch.hpp"
#include "rows.hpp"
#include "step_launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kChunk = 4096;                    // values
constexpr uint32_t kLaneVals = 8;
constexpr uint32_t kStep = kThreads * kLaneVals;     // values a workgroup takes at a time
constexpr uint32_t kMaxBlocks = 1u << 22;
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

// Values i .. i + 8 of an array of T; FULL: all of them exist, else those
// outside [0, count) are zero and are not stored.
template <typename T, bool FULL>
__device__ __forceinline__ void load8(const void* p, int64_t i, int64_t count, vec4* v) {
  if constexpr (FULL) {
#pragma unroll
    for (int j = 0; j < 8 / T::kVec; ++j) v[j] = load_vec<T>(elem<T>(p, (size_t)i) + j * T::kVec);
  } else {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = i + j >= 0 && i + j < count ? T::widen(elem<T>(p, 0)[i + j]) : 0.0f;
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
__device__ __forceinline__ void store8(void* p, int64_t i, int64_t count, const float* f) {
  if constexpr (FULL) {
#pragma unroll
    for (int j = 0; j < 8 / T::kVec; ++j) store_vec<T>(elem<T>(p, (size_t)i) + j * T::kVec, T::pack(f + j * T::kVec));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j >= 0 && i + j < count) elem<T>(p, 0)[i + j] = T::narrow(f[j]);
  }
}

typedef uint32_t codes8 __attribute__((ext_vector_type(2)));
typedef codes8 codes8_u __attribute__((aligned(1)));
template <bool FULL>
__device__ __forceinline__ codes8 load_codes(const void* p, int64_t i, int64_t count) {
  const uint8_t* q = static_cast<const uint8_t*>(p);
  if constexpr (FULL) return *reinterpret_cast<const codes8_u*>(q + i);
  codes8 v = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < count) v[j / 4] |= (uint32_t)q[i + j] << (8 * (j % 4));
  return v;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(void* p, int64_t i, int64_t count, codes8 v) {
  uint8_t* q = static_cast<uint8_t*>(p);
  if constexpr (FULL) {
    *reinterpret_cast<codes8_u*>(q + i) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < count) q[i + j] = (uint8_t)(v[j / 4] >> (8 * (j % 4)));
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

// The largest of 16 neighbouring lanes' values, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));    // lane ^ 1
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));    // lane ^ 2
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true));   // 7 - lane of 8
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, true));  // 15 - lane of 16
}

// |y| <= 448 up or down to a value that e4m3 has, up with the probability of
// what is cut off: 20 random bits are added to the word whose top 3 bits of
// mantissa stay.  Below 2^-6 the codes are evenly spaced, as they are from there
// to 2^-5, so a value is rounded there and brought back.
__device__ __forceinline__ float random_e4m3(float y, uint32_t bits16) {
  const float a = fabsf(y), lift = a < 0x1p-6f ? 0x1p-6f : 0.0f;
  float r = bits_f32((f32_bits(a + lift) + (bits16 << 4 | 8u)) & 0xFFF00000u) - lift;
  r = r > 448.0f ? 448.0f : r;
  return y == y ? copysignf(r, y) : y;
}

// x / unit rounded once, with inv = 1 / unit: the product's remainder corrects it.
__device__ __forceinline__ float quotient(float x, float unit, float inv) {
  const float q = x * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, unit, x), inv, q);
}

// Eight values of each of 16 lanes, as codes and the block's scale.
template <bool SEEDED, bool ROOT>
__device__ __forceinline__ codes8 quantise(const float* x, const uint32_t* bits, float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, f32_bits(x[j]) & 0x7FFFFFFFu);
  const float a = bits_f32(max16(top));
  const bool tiny = a < kTinyBlock;
  const float unit = a * (1.0f / 448.0f), inv = tiny ? 0.0f : 1.0f / unit;
  *scale = tiny ? 0.0f : unit;
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = quotient(x[j], unit, inv);
    if constexpr (ROOT) y[j] = x[j] > 0.0f ? (y[j] < 0x1p-9f ? 0x1p-9f : y[j]) : x[j];
    if constexpr (SEEDED) y[j] = random_e4m3(y[j], ROOT ? bits[j] >> 16 : bits[j] & 0xFFFFu);
  }
  return encode8(y);
}

// ---------------------------------------------------------------- chunks

template <typename P, typename G, int BITS, bool SEEDED, bool FULL>
__device__ __forceinline__ void chunk_body(const Tensor& t, int64_t at, const Nums& n, uint32_t key) {
  constexpr int U = kChunk / kStep;
  const int64_t count = (int64_t)t.count;
  vec4 p[U][8 / P::kVec], g[U][8 / G::kVec], m[U][2], v[U][2];
  codes8 mc[U], vc[U];
  float ms[U], vs[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = at + u * kStep + threadIdx.x * kLaneVals;
    load8<P, FULL>(t.p, i, count, p[u]);
    load8<G, FULL>(t.g, i, count, g[u]);
    if constexpr (BITS == 32) {
      load8<F32, FULL>(t.m, i, count, m[u]);
      load8<F32, FULL>(t.v, i, count, v[u]);
    } else {
      const bool there = FULL || i < count;
      mc[u] = load_codes<FULL>(t.m, i, count);
      vc[u] = load_codes<FULL>(t.v, i, count);
      ms[u] = there ? t.ms[i / HC_STATE_BLOCK] : 0.0f;
      vs[u] = there ? t.vs[i / HC_STATE_BLOCK] : 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = at + u * kStep + threadIdx.x * kLaneVals;
    float fp[8], fg[8], fm[8], fv[8], root[8];
    unpack8<P>(p[u], fp);
    unpack8<G>(g[u], fg);
    if constexpr (BITS == 32) {
      unpack8<F32>(m[u], fm);
      unpack8<F32>(v[u], fv);
    } else {
      decode8(mc[u], fm);
      decode8(vc[u], fv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        fm[j] *= ms[u];
        fv[j] *= vs[u];
        fv[j] *= fv[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fg[j] * n.c;
      fm[j] = n.b1 * fm[j] + n.a1 * x;
      fv[j] = n.b2 * fv[j] + n.a2 * (x * x);
      root[j] = __builtin_sqrtf(fv[j]);
      const float step = n.rate * fm[j] / __builtin_fmaf(root[j], n.unbias2, n.eps);
      fp[j] = __builtin_fmaf(-n.shrink * t.decay, fp[j], fp[j]) - step;
    }
    uint32_t bits[8];
    if constexpr (SEEDED) {
      // lanes of a cut chunk's first vector may lie before the tensor: they store nothing
      const uint32_t base = mix(key ^ (uint32_t)((uint64_t)i >> 32));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t lo = (uint32_t)i + j;
        // 8 values in a row may cross a multiple of 2^32 where chunks begin before the tensor
        bits[j] = mix((lo < (uint32_t)j ? mix(key ^ (uint32_t)((uint64_t)(i + j) >> 32)) : base) + lo * 0x9E3779B9u);
      }
    }
    if constexpr (SEEDED && P::kVec == 8) {
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = (f32_bits(fp[j]) + ((bits[j] * 0x9E3779B9u) >> 16)) & 0xFFFF0000u;
        r[j] = fp[j] == fp[j] ? bits_f32(w) : fp[j];
      }
      store8<P, FULL>(t.p, i, count, r);
    } else {
      store8<P, FULL>(t.p, i, count, fp);
      if constexpr (P::kVec == 4)
        if (t.copy) store8<BF16, FULL>(t.copy, i, count, fp);
    }
    if constexpr (BITS == 32) {
      store8<F32, FULL>(t.m, i, count, fm);
      store8<F32, FULL>(t.v, i, count, fv);
    } else {
      float sm, sv;
      const codes8 qm = quantise<SEEDED, false>(fm, bits, &sm), qv = quantise<SEEDED, true>(root, bits, &sv);
      store_codes<FULL>(t.m, i, count, qm);
      store_codes<FULL>(t.v, i, count, qv);
      if (i % HC_STATE_BLOCK == 0 && (FULL || i < count)) {
        t.ms[i / HC_STATE_BLOCK] = sm;
        t.vs[i / HC_STATE_BLOCK] = sv;
      }
    }
  }
}

template <typename P, typename G, int BITS, bool SEEDED>
__device__ __forceinline__ void chunk_of(const Tensor& t, int64_t at, const Nums& n, uint32_t key) {
  if (at >= 0 && at + kChunk <= (int64_t)t.count)
    chunk_body<P, G, BITS, SEEDED, true>(t, at, n, key);
  else
    chunk_body<P, G, BITS, SEEDED, false>(t, at, n, key);
}

template <int BITS, bool SEEDED>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const Tensor* tensors, const uint32_t* first, uint32_t n,
                                                         uint32_t chunks, Step s) {
  Nums nums;
  uint32_t key;
  if (!numbers(s, &nums, &key)) return;
  for (uint32_t c = blockIdx.x;;) {
    const uint32_t k = find_tensor(first, n, c);
    const Tensor t = tensors[k];
    const int64_t at = (int64_t)(c - first[k]) * kChunk - lead_of(t);
    const uint32_t own = SEEDED ? mix(key ^ (t.kind & kIndex)) : 0;
    if (t.kind & kPBf16) {
      if (t.kind & kGBf16)
        chunk_of<BF16, BF16, BITS, SEEDED>(t, at, nums, own);
      else
        chunk_of<BF16, F32, BITS, SEEDED>(t, at, nums, own);
    } else {
      if (t.kind & kGBf16)
        chunk_of<F32, BF16, BITS, SEEDED>(t, at, nums, own);
      else
        chunk_of<F32, F32, BITS, SEEDED>(t, at, nums, own);
    }
    c += gridDim.x;
    if (c < gridDim.x || c >= chunks) break;
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
    if (chunks > 0xFFFFFFFFull - kMaxBlocks) return hipErrorInvalidValue;     // 2^44 values
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
  const uint32_t grid = chunks < kMaxBlocks ? chunks : kMaxBlocks;
  auto launch = [&](auto kernel) {
    HC_ENQUEUE(kernel, grid, kThreads, stream, table, firsts, n, chunks, s);
    return hipSuccess;
  };
  if (plan.state_bits == 32) return o.seed ? launch(adamw_kernel<32, true>) : launch(adamw_kernel<32, false>);
  return o.seed ? launch(adamw_kernel<8, true>) : launch(adamw_kernel<8, false>);
}

}  // namespace hc
