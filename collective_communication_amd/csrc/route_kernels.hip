// route_kernels.hip -- each token's experts and their weights from its logits,
// and the gradient of the weights, for gfx950.
//
//   s = softmax(x) or sigmoid(x),  c = s + bias (or the order of x without one)
//   groups by their largest c or their two largest, the best of them kept;
//   the k largest c among these;  w = scale * s (/ sum of the chosen)
//
// The choice is that of 64-bit values, so that no rounding of an exponential
// decides it; nearly all of it is made by 32-bit keys whose distance from the
// values is bounded, and only what lies nearer together than that is taken in 64
// bits (about one token in 300 with 256 sigmoid scores, by its few candidates).
//
// Measured: 32,768 tokens, 256 experts, fp32 logits, a bias, 8 of 4 of 8 groups
// (35 MB) 21 us, 230 instructions a token, of which some 6 are the picks and the
// groups, 4 the 64 bits and their registers (22.5 with each pick's next largest
// searched among the lane's 16; 7 or 8 waves a SIMD instead of 6: 22.2, 21.4, with
// registers spilled); each token in 64 bits by a wave 152 us.  64 tokens, 8 of 128: 4.4 us.
#include <type_traits>

#include "lanes.hpp"
#include "launch.hpp"
#include "rows.hpp"
#include "step_launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kMaxBlocks = 1u << 22;

struct Route {
  const void* logits;
  size_t lstride;
  const float* bias;
  int32_t* experts;
  float* weights;
  const float* dweights;
  void* dlogits;
  size_t dstride;
  size_t ntokens, start;      // start: the launch's first token
  uint32_t nexperts, k, groups, group_size, top_groups, group_best, sigmoid, renormalise;
  uint32_t group_lanes;       // a power of two
  float scale;
};

// Joined over a token's LPT lanes, in all of them.
template <uint32_t LPT>
__device__ __forceinline__ uint32_t max_token(uint32_t v) {
  return join_lanes<LPT>(v, MaxOp{});
}
template <uint32_t LPT>
__device__ __forceinline__ float max_token(float v) {
  return join_lanes<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <uint32_t LPT>
__device__ __forceinline__ float sum_token(float v) {
  return join_lanes<LPT>(v, SumOp{});
}

// fp64 words that order as their values: NaN after all, 0 for what is never chosen.
__device__ __forceinline__ uint64_t order64(double c) {
  if (c != c) return ~0ull;
  c += 0.0;                                     // one zero
  const uint64_t b = (uint64_t)__double_as_longlong(c);
  return c == -__builtin_inf() ? 0 : b >> 63 ? ~b : b | 1ull << 63;
}

// The largest key of the wave and, among equal ones, the lowest id; in all lanes.
__device__ __forceinline__ void best64(uint64_t& key, uint32_t& id) {
  const uint32_t hi = (uint32_t)(key >> 32), most = max_token<64>(hi);
  const uint32_t lo = hi == most ? (uint32_t)key : 0u, least = max_token<64>(lo);
  id = ~max_token<64>(hi == most && lo == least ? ~id : 0u);
  key = (uint64_t)most << 32 | least;
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

// A wave's token in 64 bits.  Its loops stay rolled: few tokens come here, and
// the registers they would take are those of all (118 and not 80, and with
// them 4 waves a SIMD and not 6).
struct Scores64 {
  float top;
  double z;
  uint32_t sigmoid;
  __device__ __forceinline__ double operator()(float v) const {
    const double e = exp(sigmoid ? -(double)v : (double)v - top);
    return sigmoid ? 1.0 / (1.0 + e) : e / z;
  }
};
template <typename T>
__device__ __forceinline__ Scores64 scores64(const Route& r, const typename T::raw* row) {
  Scores64 s = {0.0f, 1.0, r.sigmoid};
  if (r.sigmoid) return s;
  s.top = -__builtin_inff();
#pragma unroll 1
  for (uint32_t e = lane_id(); e < r.nexperts; e += 64) s.top = fmaxf(s.top, T::widen(row[e]));
  s.top = max_token<64>(s.top);
  s.z = 0.0;
#pragma unroll 1
  for (uint32_t e = lane_id(); e < r.nexperts; e += 64) {
    const float v = T::widen(row[e]);
    if (v != -__builtin_inff()) s.z += exp((double)v - s.top);
  }
#pragma unroll 1
  for (int m = 1; m < 64; m <<= 1) s.z += __shfl_xor(s.z, m);
  return s;
}

// The token's choices, out of lanes that are `there`: expert id is its
// choice `place`.
template <typename T>
__device__ __forceinline__ void finish(const Route& r, size_t t, const typename T::raw* row, const Scores64& s, bool there,
                                       uint32_t id, uint32_t place) {
  const float v = T::widen(row[there ? id : 0]);
  const float xm = max_token<64>(there ? v : -__builtin_inff());
  float w = there ? raw_weight(r, v, s.top, (float)s.z, xm) : 0.0f;
  if (r.renormalise) {
    const float sum = sum_token<64>(w);
    if (there) w /= sum;
    if (there && s.z != s.z) w = (float)s.z;    // a NaN or an infinity among the row's logits
  }
  if (there) {
    r.experts[t * r.k + place] = (int32_t)id;
    r.weights[t * r.k + place] = w * r.scale;
  }
}

// The k largest of n <= 64 candidates, lane j's ids[j].
template <typename T>
__device__ __forceinline__ void order_candidates(const Route& r, size_t t, const uint32_t* ids, uint32_t n) {
  const uint32_t lane = lane_id();
  const typename T::raw* row = elem<T>(r.logits, t * r.lstride);
  const Scores64 s = scores64<T>(r, row);
  const uint32_t id = lane < n ? ids[lane] : 0;
  const float v = T::widen(row[id]);
  const uint64_t key = order64(r.bias ? s(v) + (double)r.bias[id] : (double)v);
  uint32_t rank = 0;
  for (uint32_t i = 0; i < n; ++i) {
    const uint64_t k = lane_read64(key, i);
    rank += k > key || (k == key && lane_read(id, i) < id);
  }
  finish<T>(r, t, row, s, lane < n && rank < r.k, id, rank);
}

// A whole token.  keys: the wave's, nexperts of them.
template <typename T>
__device__ __forceinline__ void route_token(const Route& r, size_t t, uint64_t* keys) {
  const uint32_t lane = lane_id();
  const typename T::raw* row = elem<T>(r.logits, t * r.lstride);
  const Scores64 score = scores64<T>(r, row);
#pragma unroll 1
  for (uint32_t e = lane; e < r.nexperts; e += 64) {
    const float x = T::widen(row[e]);
    double c = x;
    if (r.bias && x != -__builtin_inff()) c = score(x) + (double)r.bias[e];
    keys[e] = order64(c);
  }
  if (r.groups > 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");    // a group's experts are other lanes'
    uint64_t value = 0;
    if (lane < r.groups) {
      uint64_t a = 0, a2 = 0;           // the two largest, and where
      uint32_t ea = 0, eb = 0;
      const uint32_t from = lane * r.group_size;
#pragma unroll 4
      for (uint32_t e = from; e < from + r.group_size; ++e) {
        const uint64_t k = keys[e];
        const bool over = k > a, second = k > a2;
        a2 = over ? a : second ? k : a2;
        eb = over ? ea : second ? e : eb;
        a = over ? k : a;
        ea = over ? e : ea;
      }
      value = a;
      if (r.group_best == 2 && a) {
        double sum = 0.0;
#pragma unroll 1
        for (uint32_t i = 0; i < (a2 ? 2u : 1u); ++i) {
          const uint32_t e = i ? eb : ea;
          sum += score(T::widen(row[e])) + (r.bias ? (double)r.bias[e] : 0.0);
        }
        value = order64(sum);
      }
    }
    uint64_t kept = 0;
    for (uint32_t i = 0; i < r.top_groups; ++i) {
      uint64_t k = value;
      uint32_t g = lane;
      best64(k, g);
      if (!k) break;
      kept |= 1ull << g;
      if (lane == g) value = 0;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
    for (uint32_t e = lane; e < r.nexperts; e += 64)
      if (!(kept >> (e / r.group_size) & 1)) keys[e] = 0;
  }
  int32_t mine = -1;                    // lane j: the token's choice j
  for (uint32_t j = 0; j < r.k; ++j) {
    uint64_t k = 0;
    uint32_t id = ~0u;
#pragma unroll 2
    for (uint32_t e = lane; e < r.nexperts; e += 64) {
      const uint64_t own = keys[e];
      id = own > k ? e : id;
      k = own > k ? own : k;
    }
    best64(k, id);
    if (!k) break;
    if (lane == j) mine = (int32_t)id;
    if (id % 64 == lane) keys[id] = 0;
  }
  if (lane < r.k && mine < 0) {
    r.experts[t * r.k + lane] = -1;
    r.weights[t * r.k + lane] = 0.0f;
  }
  finish<T>(r, t, row, score, mine >= 0, (uint32_t)mine, lane);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// ---------------------------------------------------------------- many tokens in a wave

// fp32 values as words that order as they do; those below kChoosable are -inf's
// and what is not there.
constexpr uint32_t kChoosable = 0x00800000u;
__device__ __forceinline__ uint32_t order32(float c) {
  const uint32_t b = f32_bits(c);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value32(uint32_t o) {
  return bits_f32(o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}

constexpr uint32_t kMore = 8;             // candidates past the k-th

__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
  const uint32_t low = min(a, b);
  a = max(a, b);
  b = low;
}
// The four largest of V (a multiple of 4) keys, the largest first: by fours, each joined
// to those before by the larger of opposite places.
template <uint32_t V>
__device__ __forceinline__ void largest4(const uint32_t (&key)[V], uint32_t (&best)[4]) {
#pragma unroll
  for (uint32_t v = 0; v < V; v += 4) {
    uint32_t k[4] = {key[v], key[v + 1], key[v + 2], key[v + 3]};
    order(k[0], k[1]);
    order(k[2], k[3]);
    order(k[0], k[2]);
    order(k[1], k[3]);
    order(k[1], k[2]);
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) best[i] = v ? max(best[i], k[3 - i]) : k[i];
    if (v == 0) continue;
    order(best[0], best[2]);
    order(best[1], best[3]);
    order(best[0], best[1]);
    order(best[2], best[3]);
  }
}

// A token by LPT neighbouring lanes, V experts in a row each (a group by
// group_lanes of them), as 32-bit keys: the choice value's upper bits and, in
// the lowest, which of the lane's it is: a lane orders its four largest, and
// few tokens want a fifth of one lane.  Where values
// that decide are nearer than these keys and fp32's exponentials tell apart, the
// wave orders the token's candidates in 64 bits, and where these are not
// certain (groups, a NaN, many values nearly alike) takes the whole token so.
template <typename T, uint32_t LPT, uint32_t V>
__global__ void __launch_bounds__(kThreads, LPT * V <= 512 ? 6 : 1) route_kernel(Route r) {
  constexpr uint32_t N = T::kVec < V ? T::kVec : V, kTokens = kThreads / LPT;
  extern __shared__ __align__(16) uint64_t shared64[];      // as launch_route sizes it
  uint64_t* keys64 = shared64 + wave_id() * r.nexperts;
  uint32_t* slots = reinterpret_cast<uint32_t*>(shared64 + kWaves * r.nexperts);
  const uint32_t wave = wave_id(), lane = lane_id() % LPT, seg = lane_id() - lane, slot = threadIdx.x / LPT;
  const uint32_t room = r.k + kMore;
  uint32_t *ids = slots + slot * 2 * room, *keep = ids + room;
  float* chosen_x = reinterpret_cast<float*>(slots + kTokens * 2 * room) + slot * r.k;
  const uint32_t g = lane / r.group_lanes, in_group = lane % r.group_lanes;
  const uint32_t n = g < r.groups && in_group * V < r.group_size ? min(V, r.group_size - in_group * V) : 0;
  const uint32_t e0 = n ? g * r.group_size + in_group * V : 0;
  const bool by_score = r.bias != nullptr;                      // else by the logits themselves
  const bool softmax = !r.sigmoid;
  const bool need_z = softmax && (by_score || !r.renormalise || (r.groups > 1 && r.group_best == 2));
  const bool exact = !by_score && T::kVec == 8;                 // bf16 logits keep all their bits in a key
  const size_t first = r.start + (size_t)blockIdx.x * kTokens;
  const bool live = first + slot < r.ntokens;
  const size_t t = live ? first + slot : r.ntokens - 1;
  const typename T::raw* row = elem<T>(r.logits, t * r.lstride);
  float x[V];
  if (n == V) {
    if constexpr (N == T::kVec) {
#pragma unroll
      for (uint32_t v = 0; v < V; v += N) T::unpack(load_vec<T>(row + e0 + v), x + v);
    } else {
      typedef uint32_t vec2_u __attribute__((ext_vector_type(2), aligned(2)));
      const vec2_u w = *reinterpret_cast<const vec2_u*>(row + e0);      // 4 bf16
#pragma unroll
      for (uint32_t v = 0; v < 2; ++v) {
        x[2 * v] = bits_f32(w[v] << 16);
        x[2 * v + 1] = bits_f32(w[v] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (uint32_t v = 0; v < V; ++v) x[v] = T::widen(row[e0 + (v < n ? v : 0)]);
#pragma unroll
    for (uint32_t v = 0; v < V; ++v) x[v] = v < n ? x[v] : -__builtin_inff();
  }
  float top = 0.0f, z = 1.0f;
  uint32_t key[V];
  bool odd = false;          // a value for the 64 bits
  if (need_z) {
    top = x[0];
#pragma unroll
    for (uint32_t v = 1; v < V; ++v) top = fmaxf(top, x[v]);
    top = max_token<LPT>(top);
    const float from = top == -__builtin_inff() ? 0.0f : top;
    z = 0.0f;
#pragma unroll
    for (uint32_t v = 0; v < V; ++v) {
      const float e = expf(x[v] - from);
      z += e;
      if (by_score) key[v] = f32_bits(e);
    }
    z = sum_token<LPT>(z);
    odd = z != z;
  }
  if (by_score) {
    float b[V];
    if (n == V) {
#pragma unroll
      for (uint32_t v = 0; v < V; v += 4) F32::unpack(load_vec<F32>(elem<F32>(r.bias, e0 + v)), b + v);
    } else {
#pragma unroll
      for (uint32_t v = 0; v < V; ++v) b[v] = r.bias[e0 + (v < n ? v : 0)];
    }
    // fast scores here: the distances that decide are checked below
    float c[V];
    if (softmax) {
      const float per = __builtin_amdgcn_rcpf(z);
#pragma unroll
      for (uint32_t v = 0; v < V; ++v) c[v] = bits_f32(key[v]) * per;
    } else {
#pragma unroll
      for (uint32_t v = 0; v < V; ++v)
        c[v] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[v] * -1.44269504f));
    }
#pragma unroll
    for (uint32_t v = 0; v < V; ++v) {
      const float sum = c[v] + b[v];
      key[v] = order32(x[v] == -__builtin_inff() ? x[v] : sum);
    }
  } else {
#pragma unroll
    for (uint32_t v = 0; v < V; ++v) key[v] = order32(x[v] + 0.0f);      // one zero
  }
  uint32_t lowest = key[0], highest = key[0];
#pragma unroll
  for (uint32_t v = 1; v < V; ++v) {
    lowest = min(lowest, key[v]);
    highest = max(highest, key[v]);
  }
  // a NaN is above infinity or below its negative: for the 64 bits
  odd = odd || lowest < order32(-__builtin_inff()) || highest > order32(__builtin_inff());
#pragma unroll
  for (uint32_t v = 0; v < V; ++v) key[v] = (key[v] & ~(V - 1)) | (V - 1 - v);
  // How far a value's key may be from it: what the key cuts off and a sum's
  // rounding, relative to it, and the score's own error, in halves of an ulp, 2^-24.
  // An exponential of x is off by |x| + 2 of them, and (|x| + 2) e^-|x| is at most 2.
  // A sigmoid: |x| s (1 - s) is below 0.3, and s (1 - s) at most 1/4, with the
  // argument's constant, its sum and its quotient below 8; 16 are taken.
  // A softmax, relative to the largest that there can be, 1 / z: the exponential 2
  // and the product 1 for each of two that are compared, and for both together the
  // reciprocal 2 and z, by V - 1 sums in turn, 6 over the lanes and its exponentials'
  // 2 and mean |x|, which for 1024 experts is below 4.5: V + 20 for two, V / 2 + 10
  // for one; V / 2 + 12 are taken, and 16 at least.
  constexpr float kCut = V * 0x1p-23f, kSoft = V > 8 ? V / 2 + 12 : 16;
  const float unit = softmax ? kSoft * 0x1p-24f / z : 0x1p-20f;
  auto off = [=](float c) { return fabsf(c) * (kCut + 0x1p-23f) + unit; };
  uint32_t top4[4];
  largest4<V>(key, top4);
  // a lane's largest key up to `limit`, for the few that four are not enough for
  auto largest = [&](uint32_t limit) {
    uint32_t d = limit;
#pragma unroll
    for (uint32_t v = 0; v < V; ++v) d = min(d, limit - key[v]);     // wraps far up for those above
    return limit - d;
  };
  if (r.groups > 1) {
    // the two largest keys of the lane's group
    uint32_t a = top4[0], b = top4[1];
    for (uint32_t m = 1; m < r.group_lanes; m <<= 1) {
      const uint32_t a2 = (uint32_t)__shfl_xor((int)a, (int)m), b2 = (uint32_t)__shfl_xor((int)b, (int)m);
      b = max(max(b, b2), min(a, a2));
      a = max(a, a2);
    }
    const bool any = a >= kChoosable;
    float value = value32(a & ~(V - 1)), near = 0.0f;
    if (r.group_best == 2) {
      float va = value, vb = value32(b & ~(V - 1));
      if (!by_score) {
        va = softmax ? expf(va - top) / z : 1.0f / (1.0f + expf(-va));
        vb = softmax ? expf(vb - top) / z : 1.0f / (1.0f + expf(-vb));
      }
      if (b < kChoosable) vb = 0.0f;
      value = va + vb;
      near = off(va) + off(vb);
      // the bits that a logit's key lacks move its score by as much as it is large
      if (!by_score) near += kCut * (fabsf(va * value32(a)) + (b < kChoosable ? 0.0f : fabsf(vb * value32(b))));
    } else if (by_score) {
      near = off(value);
    }
    if (!any) value = -__builtin_inff();
    auto rank_of = [&](auto own) {
      uint32_t rank = 0;
      for (uint32_t o = 0; o < r.groups; ++o) {
        const auto other = __shfl(own, (int)(seg + o * r.group_lanes));
        rank += other > own || (other == own && o < g);
      }
      return rank;
    };
    uint32_t rank = rank_of(value);
    bool kept = any && rank < r.top_groups;
    // the worst that stays against the best that goes
    const float low = -max_token<LPT>(kept ? -value : -__builtin_inff());
    const float high = max_token<LPT>(any && !kept ? value : -__builtin_inff());
    const float margin = 2.0f * max_token<LPT>(any ? near : 0.0f);
    const bool close = !(exact && r.group_best == 1) && high > -__builtin_inff() && !(low - high > margin);
    if (__any(close && live)) {
      // the groups' values in 64 bits, of each lane's two largest; where its third
      // may be among them, or with a row's sum to take, the whole token
      const float c2 = value32(top4[1] & ~(V - 1)), c3 = value32(top4[2] & ~(V - 1));
      const bool sure = top4[2] < kChoosable || c2 - c3 > 2.0f * (near + off(c2));
      auto exactly = [&](uint32_t k) {
        const uint32_t e = e0 + (k >= kChoosable ? (V - 1) - (k & (V - 1)) : 0);
        const double v = T::widen(row[e]);
        const double s = by_score || r.group_best == 2 ? 1.0 / (1.0 + exp(-v)) + (by_score ? (double)r.bias[e] : 0.0) : v;
        return k >= kChoosable ? s : -__builtin_inf();
      };
      double d = exactly(top4[0]), d2 = exactly(top4[1]);
      if (d2 > d) {
        const double swap = d;
        d = d2;
        d2 = swap;
      }
      for (uint32_t m = 1; m < r.group_lanes; m <<= 1) {
        const double o = __shfl_xor(d, (int)m), o2 = __shfl_xor(d2, (int)m);
        d2 = fmax(fmax(d2, o2), fmin(d, o));
        d = fmax(d, o);
      }
      if (r.group_best == 2 && d2 > -__builtin_inf()) d += d2;
      rank = rank_of(d);
      if (close) {
        kept = any && rank < r.top_groups;
        if (softmax || !sure) odd = true;
      }
    }
    if (!kept) top4[0] = 0;                 // never taken, and so none after it
  }
  // the k largest, and those after that may belong to them
  const uint32_t picks = exact ? r.k : r.k + kMore;
  uint32_t found = 0, before = 0;
  bool open = !exact;        // whether the next may still belong to them
  for (uint32_t j = 0; j < picks; ++j) {
    const uint32_t best = top4[0], m = max_token<LPT>(best);
    const bool there = m >= kChoosable;
    if (j >= r.k) {
      const float c = value32(before & ~(V - 1)), c2 = value32(m & ~(V - 1));
      open = open && there && !(c - c2 > (by_score ? off(c) + off(c2) : 0.0f));
      if (!__any(open && live)) break;
    }
    const bool take = there && (j < r.k || open);
    const uint64_t same = __ballot(take && (best | (V - 1)) == (m | (V - 1)));
    if (!same) break;
    uint32_t winner;
    if constexpr (LPT == 64)
      winner = (uint32_t)__builtin_ctzll(same);
    else if constexpr (LPT == 32)
      winner = (uint32_t)__builtin_ctz(seg ? (uint32_t)(same >> 32) : (uint32_t)same);
    else
      winner = (uint32_t)__builtin_ctz((seg < 32 ? (uint32_t)same : (uint32_t)(same >> 32)) >> (seg & 31));
    found += take;
    before = m;
    if (take && winner == lane) {
      ids[j] = e0 + (V - 1) - (best & (V - 1));
      keep[j] = best;
      top4[0] = top4[1];
      top4[1] = top4[2];
      top4[2] = top4[3];
      top4[3] = 0;
      if (V > 4 && top4[0] == 0) top4[0] = largest(best - 1);
    }
  }
  // more candidates than there was room for, or than a wave has lanes
  if ((open && found == r.k + kMore) || found > 64) odd = true;
  constexpr uint64_t kLanes = LPT == 64 ? ~0ull : (1ull << (LPT & 63)) - 1;
  const bool whole = __ballot(odd) >> seg & kLanes;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  // the chosen logits, and whether each is far enough before the next
  float xm = -__builtin_inff();
  const uint32_t chosen = min(found, r.k);
  bool again = whole || found > chosen;
  for (uint32_t j = lane; j < chosen; j += LPT) {
    const uint32_t e = ids[j];
    const float v = T::widen(row[e]);
    chosen_x[j] = v;
    xm = fmaxf(xm, v);
    if (!exact && j + 1 < chosen) {
      const float c = value32(keep[j] & ~(V - 1)), c2 = value32(keep[j + 1] & ~(V - 1));
      if (!(c - c2 > (by_score ? off(c) + off(c2) : 0.0f))) {
        const uint32_t e2 = ids[j + 1];     // the same value in the order of experts is right
        again = again || f32_bits(v) != f32_bits(T::widen(row[e2])) ||
                (by_score && f32_bits(r.bias[e]) != f32_bits(r.bias[e2]));
      }
    }
  }
  xm = max_token<LPT>(xm);
  float sum = 0.0f;
  if (r.renormalise) {
    for (uint32_t j = lane; j < chosen; j += LPT) sum += raw_weight(r, chosen_x[j], top, z, xm);
    sum = sum_token<LPT>(sum);
  }
  uint64_t redo = __ballot(again && live);
  if (live && !(redo >> seg & kLanes)) {
    for (uint32_t j = lane; j < r.k; j += LPT) {
      float w = 0.0f;
      if (j < chosen) {
        w = raw_weight(r, chosen_x[j], top, z, xm);
        if (r.renormalise) w /= sum;
      }
      r.experts[t * r.k + j] = j < chosen ? (int32_t)ids[j] : -1;
      r.weights[t * r.k + j] = w * r.scale;
    }
  }
  while (redo) {
    const uint32_t at = (uint32_t)__builtin_ctzll(redo) / LPT;         // which of the wave's tokens
    const uint32_t of = wave * (64 / LPT) + at, n = lane_read(found, at * LPT);
    if (lane_read(whole, at * LPT) || n < r.k)
      route_token<T>(r, first + of, keys64);
    else
      order_candidates<T>(r, first + of, slots + of * 2 * room, n);
    redo &= ~(kLanes << (at * LPT));
  }
}

// ---------------------------------------------------------------- gradient

// A token by LPT neighbouring lanes: its row of gradients is made in shared memory,
// the few slots' on top of zeroes (or of the softmax's share), and goes out by
// vectors.  Shared memory holds a token's row and three words of each slot, as
// many as there are, so that all of a CU's waves find room.
// Measured: 32,768 tokens, 8 of 256 experts, fp32 (37 MB) 11.2 us; 9999 tokens,
// 4 of 60, bf16, the whole softmax's 6.0 us.
constexpr uint32_t kGradVals = 16;      // experts a lane, at least
__host__ __device__ __forceinline__ uint32_t grad_row(uint32_t nexperts) { return (nexperts + 3) & ~3u; }
template <typename T, uint32_t LPT>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(Route r) {
  constexpr uint32_t N = T::kVec, kTokens = kThreads / LPT;
  extern __shared__ __align__(16) float shared[];
  const uint32_t lane = threadIdx.x % LPT, slot = threadIdx.x / LPT, width = grad_row(r.nexperts);
  float* row = shared + slot * width;
  int32_t* id = reinterpret_cast<int32_t*>(shared + kTokens * width) + slot * r.k;
  float* val = shared + kTokens * (width + r.k) + slot * r.k;
  float* raw = shared + kTokens * (width + 2 * r.k) + slot * r.k;
  const bool dense = !r.renormalise && !r.sigmoid;
  const size_t first = r.start + (size_t)blockIdx.x * kTokens;
  const bool live = first + slot < r.ntokens;
  const size_t t = live ? first + slot : r.ntokens - 1;
  const typename T::raw* x = elem<T>(r.logits, t * r.lstride);
  // the chosen logits
  float xm = -__builtin_inff();
  for (uint32_t j = lane; j < r.k; j += LPT) {
    const int32_t e = r.experts[t * r.k + j];
    const float dw = r.dweights[t * r.k + j];
    const bool in = (uint32_t)e < r.nexperts;
    const float v = T::widen(x[in ? e : 0]);
    const bool there = in && v != -__builtin_inff();
    id[j] = there ? e : -1;
    val[j] = there ? dw * r.scale : 0.0f;
    raw[j] = v;
    if (there) xm = fmaxf(xm, v);
  }
  // the row's softmax, where its gradient reaches every expert
  float top = -__builtin_inff(), z = 0.0f;
  if (dense) {
    for (uint32_t e = lane; e < r.nexperts; e += LPT) {
      row[e] = T::widen(x[e]);
      top = fmaxf(top, row[e]);
    }
    top = max_token<LPT>(top);
    for (uint32_t e = lane; e < r.nexperts; e += LPT) {
      row[e] = row[e] == -__builtin_inff() ? 0.0f : expf(row[e] - top);
      z += row[e];
    }
    z = sum_token<LPT>(z);
  } else {
    for (uint32_t e = lane * 4; e < width; e += LPT * 4) *reinterpret_cast<vec4*>(row + e) = vec4{0, 0, 0, 0};
  }
  xm = max_token<LPT>(xm);
  float sum = 0.0f, dot = 0.0f;
  for (uint32_t j = lane; j < r.k; j += LPT) {
    if (id[j] < 0) continue;
    const float v = raw[j], a = raw_weight(r, v, top, z, xm);
    sum += a;
    raw[j] = a;
  }
  if (r.renormalise) sum = sum_token<LPT>(sum);
  // shares first, so that a single one is 1 and its gradient 0
  for (uint32_t j = lane; j < r.k; j += LPT) {
    if (id[j] < 0) continue;
    if (r.renormalise) raw[j] /= sum;
    dot = __builtin_fmaf(raw[j], val[j], dot);
  }
  dot = sum_token<LPT>(dot);
  // d/dx of each slot, with 1 - sigmoid(x)
  for (uint32_t j = lane; j < r.k; j += LPT) {
    const int32_t e = id[j];
    if (e < 0) continue;
    const float d = raw[j] * (r.renormalise ? val[j] - dot : val[j]);
    val[j] = r.sigmoid ? d / (1.0f + expf(T::widen(x[e]))) : d;
  }
  if (dense) {
    const float share = z == 0.0f ? 0.0f : -dot / z;
    for (uint32_t e = lane; e < r.nexperts; e += LPT) row[e] *= share;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  // an expert listed twice is added up, in slot order, by its first slot
  for (uint32_t j = lane; j < r.k; j += LPT) {
    const int32_t e = id[j];
    if (e < 0) continue;
    float d = 0.0f;
    bool mine = true;
#pragma unroll 4
    for (uint32_t i = 0; i < r.k; ++i) {
      const bool same = id[i] == e;
      mine = mine && !(same && i < j);
      d += same ? val[i] : 0.0f;
    }
    if (mine) row[e] += d;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (!live) return;
  typename T::raw* out = elem<T>(r.dlogits, t * r.dstride);
  for (uint32_t c = lane * N; c < r.nexperts; c += LPT * N) {
    if (c + N <= r.nexperts) {
      float f[N];
#pragma unroll
      for (uint32_t i = 0; i < N; i += 4) {
        const vec4 w = *reinterpret_cast<const vec4*>(row + c + i);
        F32::unpack(w, f + i);
      }
      store_vec<T>(out + c, T::pack(f));
    } else {
      for (uint32_t e = c; e < r.nexperts; ++e) out[e] = T::narrow(row[e]);
    }
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
  // the fewest values a lane whose lanes are enough: 4 up to 16 of them, 16 up
  // to a wave (32 only for groups just above a multiple of 16)
  auto lanes = [&](uint32_t v) {
    r.group_lanes = 1;
    while (r.group_lanes * v < r.group_size) r.group_lanes *= 2;
    uint32_t all = r.group_lanes;
    while (all < r.groups * r.group_lanes) all *= 2;
    return all;
  };
  auto run = [&](auto lpt, auto vals) {
    constexpr uint32_t LPT = decltype(lpt)::value, V = decltype(vals)::value;
    // a wave's experts in 64 bits, and of each token candidates, keys and chosen logits
    const uint32_t lds = 8 * kWaves * nexperts + 4 * (kThreads / LPT) * (2 * (r.k + kMore) + r.k);
    for (r.start = 0; r.start < ntokens; r.start += (size_t)kMaxBlocks * (kThreads / LPT)) {
      const uint32_t blocks = blocks_for(ntokens - r.start, kThreads / LPT);
      const hipError_t e = dtype == HC_F32 ? enqueue_lds(lds, route_kernel<F32, LPT, V>, blocks, kThreads, stream, r)
                                           : enqueue_lds(lds, route_kernel<BF16, LPT, V>, blocks, kThreads, stream, r);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  // 64 tokens of up to 16 experts, or 4 of HC_MAX_EXPERTS
  static_assert(8 * kWaves * 16 + 4 * 64 * (3 * HC_MAX_TOPK + 2 * kMore) <= 64 << 10 &&
                    8 * kWaves * HC_MAX_EXPERTS + 4 * 32 * (3 * HC_MAX_TOPK + 2 * kMore) <= 64 << 10,
                "shared memory of a workgroup");
#define HC_LANES(L, V) run(std::integral_constant<uint32_t, L>{}, std::integral_constant<uint32_t, V>{})
  uint32_t n = lanes(4);
  if (n <= 4) return HC_LANES(4, 4);
  if (n <= 8) return HC_LANES(8, 4);
  if (n <= 16) return HC_LANES(16, 4);
  n = lanes(16);
  if (n <= 8) return HC_LANES(8, 16);
  if (n <= 16) return HC_LANES(16, 16);
  if (n <= 32) return HC_LANES(32, 16);
  if (n <= 64) return HC_LANES(64, 16);
  lanes(32);
  return HC_LANES(64, 32);
#undef HC_LANES
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
    constexpr uint32_t LPT = decltype(lanes)::value, kTokens = kThreads / LPT;
    static_assert(4 * kTokens * (LPT * kGradVals + 3 * HC_MAX_TOPK) <= 64 << 10, "shared memory of a workgroup");
    const uint32_t lds = 4 * kTokens * (grad_row(nexperts) + 3 * r.k);
    for (r.start = 0; r.start < ntokens; r.start += (size_t)kMaxBlocks * kTokens) {
      const uint32_t blocks = blocks_for(ntokens - r.start, kTokens);
      const hipError_t e = dtype == HC_F32
                               ? enqueue_lds(lds, route_grad_kernel<F32, LPT>, blocks, kThreads, stream, r)
                               : enqueue_lds(lds, route_grad_kernel<BF16, LPT>, blocks, kThreads, stream, r);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  if (nexperts <= 8 * kGradVals) return run(std::integral_constant<uint32_t, 8>{});
  if (nexperts <= 16 * kGradVals) return run(std::integral_constant<uint32_t, 16>{});
  if (nexperts <= 32 * kGradVals) return run(std::integral_constant<uint32_t, 32>{});
  return run(std::integral_constant<uint32_t, 64>{});
}

}  // namespace hc
