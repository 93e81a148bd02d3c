// route_kernels.hip -- each token's experts and their weights from its logits,
// and the gradient of the weights, for gfx950.
//
//   s = softmax(x) or sigmoid(x),  c = s + bias (or the order of x without one)
//   groups by their largest c or their two largest, the best of them kept;
//   the k largest c among these;  w = scale * s (/ sum of the chosen)
//
// The choice is made on 64-bit values, so that no rounding of an exponential
// decides it.
#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"
#include "step_launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kMaxBlocks = 1u << 22;
constexpr uint32_t kMaxExperts = HC_MAX_EXPERTS;

struct Route {
  const void* logits;
  size_t lstride;
  const float* bias;
  int32_t* experts;
  float* weights;
  const float* dweights;
  void* dlogits;
  size_t dstride;
  size_t ntokens;
  uint32_t nexperts, k, groups, group_size, top_groups, group_best, sigmoid, renormalise;
  float scale;
};

// fp64 words that order as their values: NaN after all, 0 for what is never chosen.
__device__ __forceinline__ uint64_t order64(double c) {
  if (c != c) return ~0ull;
  c += 0.0;                                     // one zero
  const uint64_t b = (uint64_t)__double_as_longlong(c);
  return c == -__builtin_inf() ? 0 : b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int m) {
  return (uint64_t)(uint32_t)__shfl_xor((int)(x >> 32), m) << 32 | (uint32_t)__shfl_xor((int)(uint32_t)x, m);
}
__device__ __forceinline__ double shfl_xor_f64(double x, int m) {
  return __longlong_as_double((long long)shfl_xor64((uint64_t)__double_as_longlong(x), m));
}

// The largest key of the wave and, among equal ones, the lowest id; in all lanes.
__device__ __forceinline__ void best64(uint64_t& key, uint32_t& id) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint64_t k2 = shfl_xor64(key, m);
    const uint32_t i2 = (uint32_t)__shfl_xor((int)id, m);
    if (k2 > key || (k2 == key && i2 < id)) {
      key = k2;
      id = i2;
    }
  }
}

// The weight of one chosen logit out of `lanes` neighbouring lanes' (the others'
// there is false).  A renormalised one comes from the chosen logits alone, by
// their distance from the largest, so that no score vanishes first.
__device__ __forceinline__ float raw_weight(const Route& r, float x, float top, float z, float xm) {
  if (!r.renormalise) return r.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - top) / z;
  if (!r.sigmoid) return expf(x - xm);
  if (x > 0.0f) return 1.0f / (1.0f + expf(-x));
  return expf(x - fminf(xm, 0.0f)) / (1.0f + expf(x));
}

// One token by one wave, in 64 bits.  keys: the wave's, nexperts of them.
template <typename T>
__device__ void route_token(const Route& r, size_t t, uint64_t* keys) {
  const uint32_t lane = lane_id();
  const typename T::raw* x = elem<T>(r.logits, t * r.lstride);
  double top = -__builtin_inf(), z = 0.0;
  if (!r.sigmoid) {
    for (uint32_t e = lane; e < r.nexperts; e += 64) {
      const double v = T::widen(x[e]);
      top = v > top ? v : top;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double o = shfl_xor_f64(top, m);
      top = o > top ? o : top;
    }
    for (uint32_t e = lane; e < r.nexperts; e += 64) {
      const double v = T::widen(x[e]);
      if (v != -__builtin_inf()) z += exp(v - top);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) z += shfl_xor_f64(z, m);
  }
  auto score = [&](double v) { return r.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - top) / z; };
  auto choice = [&](uint32_t e) {
    const double v = T::widen(x[e]);
    if (!r.bias || v == -__builtin_inf()) return v;
    return score(v) + (double)r.bias[e];
  };
  for (uint32_t e = lane; e < r.nexperts; e += 64) keys[e] = order64(choice(e));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");    // a group's experts are other lanes'
  if (r.groups > 1) {
    uint64_t key = 0;
    if (lane < r.groups) {
      uint64_t a = 0, b = 0;            // the two largest, and where
      uint32_t ea = 0, eb = 0;
      for (uint32_t e = lane * r.group_size; e < (lane + 1) * r.group_size; ++e) {
        const uint64_t k = keys[e];
        if (k > a) {
          b = a;
          eb = ea;
          a = k;
          ea = e;
        } else if (k > b) {
          b = k;
          eb = e;
        }
      }
      key = a;
      if (r.group_best == 2 && a) {
        auto value = [&](uint32_t e) { return r.bias ? choice(e) : score(T::widen(x[e])); };
        key = order64(value(ea) + (b ? value(eb) : 0.0));
      }
    }
    uint64_t kept = 0;
    for (uint32_t i = 0; i < r.top_groups; ++i) {
      uint64_t k = key;
      uint32_t g = lane;
      best64(k, g);
      if (!k) break;
      kept |= 1ull << g;
      if (lane == g) key = 0;
    }
    for (uint32_t e = lane; e < r.nexperts; e += 64)
      if (!(kept >> (e / r.group_size) & 1)) keys[e] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  int32_t mine = -1;                    // lane j: the token's choice j
  for (uint32_t j = 0; j < r.k; ++j) {
    uint64_t key = 0;
    uint32_t id = ~0u;
    for (uint32_t e = lane; e < r.nexperts; e += 64)
      if (keys[e] > key) {
        key = keys[e];
        id = e;
      }
    best64(key, id);
    if (!key) break;
    if (lane == j) mine = (int32_t)id;
    if (id % 64 == lane) keys[id] = 0;
  }
  const bool there = mine >= 0;
  const float v = there ? T::widen(x[mine]) : 0.0f;
  float xm = there ? v : -__builtin_inff();
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) xm = fmaxf(xm, __shfl_xor(xm, m));
  float w = there ? raw_weight(r, v, (float)top, (float)z, xm) : 0.0f;
  if (r.renormalise) {
    float sum = w;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if (there) w /= sum;
    if (there && z != z) w = (float)z;          // a NaN or an infinity among the row's logits
  }
  if (lane < r.k) {
    r.experts[t * r.k + lane] = mine;
    r.weights[t * r.k + lane] = w * r.scale;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) route_kernel(Route r) {
  __shared__ uint64_t keys[kWaves][kMaxExperts];
  const uint32_t wave = wave_id();
  for (size_t t = (size_t)blockIdx.x * kWaves + wave; t < r.ntokens; t += (size_t)gridDim.x * kWaves)
    route_token<T>(r, t, keys[wave]);
}

// ---------------------------------------------------------------- gradient

// A token by LPT neighbouring lanes: its row of gradients is made in LDS, the
// few slots' on top of zeroes (or of the softmax's share), and goes out by vectors.
template <typename T, uint32_t LPT>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(Route r) {
  constexpr uint32_t N = T::kVec, V = 16, kTokens = kThreads / LPT;
  __shared__ __align__(16) float rows[kTokens][LPT * V];
  __shared__ int32_t ids[kTokens][HC_MAX_TOPK];
  __shared__ float vals[kTokens][HC_MAX_TOPK];
  const uint32_t lane = threadIdx.x % LPT, slot = threadIdx.x / LPT;
  float* row = rows[slot];
  int32_t* id = ids[slot];
  float* val = vals[slot];
  auto join = [&](float v) {
#pragma unroll
    for (uint32_t m = 1; m < LPT; m <<= 1) v += __shfl_xor(v, (int)m);
    return v;
  };
  auto most = [&](float v) {
#pragma unroll
    for (uint32_t m = 1; m < LPT; m <<= 1) v = fmaxf(v, __shfl_xor(v, (int)m));
    return v;
  };
  const bool dense = !r.renormalise && !r.sigmoid;
  for (size_t first = (size_t)blockIdx.x * kTokens; first < r.ntokens; first += (size_t)gridDim.x * kTokens) {
    const bool live = first + slot < r.ntokens;
    const size_t t = live ? first + slot : r.ntokens - 1;
    const typename T::raw* x = elem<T>(r.logits, t * r.lstride);
    // the row's softmax, where its gradient reaches every expert
    float top = -__builtin_inff(), z = 0.0f;
    if (dense) {
      for (uint32_t e = lane; e < r.nexperts; e += LPT) top = fmaxf(top, T::widen(x[e]));
      top = most(top);
      for (uint32_t e = lane; e < r.nexperts; e += LPT) {
        const float v = T::widen(x[e]);
        row[e] = v == -__builtin_inff() ? 0.0f : expf(v - top);
        z += row[e];
      }
      z = join(z);
    } else {
      for (uint32_t e = lane * 4; e < LPT * V; e += LPT * 4) *reinterpret_cast<vec4*>(row + e) = vec4{0, 0, 0, 0};
    }
    // the chosen logits
    float xm = -__builtin_inff();
    for (uint32_t j = lane; j < r.k; j += LPT) {
      const int32_t e = r.experts[t * r.k + j];
      const bool there = (uint32_t)e < r.nexperts && T::widen(x[e]) != -__builtin_inff();
      id[j] = there ? e : -1;
      val[j] = there ? r.dweights[t * r.k + j] * r.scale : 0.0f;
      if (there) xm = fmaxf(xm, T::widen(x[e]));
    }
    xm = most(xm);
    float sum = 0.0f, dot = 0.0f;
    for (uint32_t j = lane; j < r.k; j += LPT) {
      if (id[j] < 0) continue;
      const float a = raw_weight(r, T::widen(x[id[j]]), top, z, xm);
      sum += a;
      dot = __builtin_fmaf(a, val[j], dot);
    }
    sum = join(sum);
    dot = join(dot);
    // d/dx of each slot
    for (uint32_t j = lane; j < r.k; j += LPT) {
      if (id[j] < 0) continue;
      const float v = T::widen(x[id[j]]), a = raw_weight(r, v, top, z, xm);
      float d = r.renormalise ? a / sum * (val[j] - dot / sum) : a * val[j];
      if (r.sigmoid) d *= 1.0f / (1.0f + expf(v));       // 1 - sigmoid(v)
      val[j] = d;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (dense)
      for (uint32_t e = lane; e < r.nexperts; e += LPT) row[e] *= z == 0.0f ? 0.0f : -dot / z;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // an expert listed twice is added up, in slot order, by its first slot
    for (uint32_t j = lane; j < r.k; j += LPT) {
      const int32_t e = id[j];
      if (e < 0) continue;
      float d = 0.0f;
      bool mine = true;
      for (uint32_t i = 0; i < r.k; ++i)
        if (id[i] == e) {
          mine = mine && i >= j;
          d += val[i];
        }
      if (mine) row[e] += d;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (live) {
      typename T::raw* out = elem<T>(r.dlogits, t * r.dstride);
      for (uint32_t c = lane * N; c < r.nexperts; c += LPT * N) {
        float f[N];
        if (c + N <= r.nexperts) {
#pragma unroll
          for (uint32_t i = 0; i < N; ++i) f[i] = row[c + i];
          store_vec<T>(out + c, T::pack(f));
        } else {
          for (uint32_t e = c; e < r.nexperts; ++e) out[e] = T::narrow(row[e]);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

Route route_of(const void* logits, size_t ntokens, uint32_t nexperts, size_t lstride, const hc_route_opts_t& o) {
  Route r = {};
  r.logits = logits;
  r.lstride = lstride;
  r.ntokens = ntokens;
  r.nexperts = nexperts;
  r.bias = o.bias;
  r.k = (uint32_t)o.k;
  r.groups = (uint32_t)o.ngroups;
  r.group_size = r.groups ? nexperts / r.groups : nexperts;
  r.top_groups = (uint32_t)o.top_groups;
  r.group_best = (uint32_t)o.group_best;
  r.sigmoid = o.scores == HC_SCORES_SIGMOID;
  r.renormalise = o.renormalise != 0;
  r.scale = o.scale;
  return r;
}

inline uint32_t blocks_for(uint64_t tokens, uint32_t per_block) {
  const uint64_t b = (tokens + per_block - 1) / per_block;
  return (uint32_t)(b < kMaxBlocks ? b : kMaxBlocks);
}

}  // namespace

hipError_t launch_route(const void* logits, hc_dtype_t dtype, size_t ntokens, uint32_t nexperts, size_t lstride,
                        const hc_route_opts_t& o, int32_t* experts, float* weights, hipStream_t stream) {
  Route r = route_of(logits, ntokens, nexperts, lstride, o);
  r.experts = experts;
  r.weights = weights;
  if (dtype == HC_F32)
    HC_ENQUEUE(route_kernel<F32>, blocks_for(ntokens, kWaves), kThreads, stream, r);
  else
    HC_ENQUEUE(route_kernel<BF16>, blocks_for(ntokens, kWaves), kThreads, stream, r);
  return hipSuccess;
}

hipError_t launch_route_grad(const void* logits, hc_dtype_t dtype, size_t ntokens, uint32_t nexperts, size_t lstride,
                             const hc_route_opts_t& o, const int32_t* experts, const float* dweights, void* dlogits,
                             size_t dstride, hipStream_t stream) {
  Route r = route_of(logits, ntokens, nexperts, lstride, o);
  r.experts = const_cast<int32_t*>(experts);    // only read
  r.dweights = dweights;
  r.dlogits = dlogits;
  r.dstride = dstride;
  auto run = [&](auto lanes) {
    constexpr uint32_t LPT = decltype(lanes)::value;
    const uint32_t blocks = blocks_for(ntokens, kThreads / LPT);
    if (dtype == HC_F32)
      HC_ENQUEUE((route_grad_kernel<F32, LPT>), blocks, kThreads, stream, r);
    else
      HC_ENQUEUE((route_grad_kernel<BF16, LPT>), blocks, kThreads, stream, r);
    return hipSuccess;
  };
  if (nexperts <= 128) return run(std::integral_constant<uint32_t, 8>{});
  if (nexperts <= 256) return run(std::integral_constant<uint32_t, 16>{});
  if (nexperts <= 512) return run(std::integral_constant<uint32_t, 32>{});
  return run(std::integral_constant<uint32_t, 64>{});
}

}  // namespace hc
