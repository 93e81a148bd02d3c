// norm_kernels.hip -- the root-mean-square norm of rows after a residual's
// addition, with rows of their own type or of 8 bits, and its gradient, for
// gfx950.
//
//   h = round(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = round(h r w)
//   8 bits: t = h w, a = largest |t| of a group, q = e4m3(t (448 / a)), scale = a r / 448
//   dx = round(r (dy w - h r^2 mean(dy w h)) + dsum),  dw = sum over rows of dy h r
//
// All are streams over rows: a row is loaded once into the registers of as many
// lanes as its width has vectors for (8 to 64 of a wave, or 4, 8 or 16 waves), its
// sums are joined there, and it is written from there.  The gradient of the
// weight is summed over a workgroup's rows in registers and left as one row of
// partials per workgroup, which a second launch adds in a fixed order.
//
// Measured (a large copy reaches 4.8-5.2 TB/s here): 16,384 x 4096 bf16 with a residual
// to 8 bits, a scale for 128 columns (472 MB) 93 us, 5.1 TB/s (105 with plain
// stores and joins through shared memory, 111 by 8 waves a row, 126 by 2); 60,000 x
// 2048 without a residual, which is bound by the lanes' work, 103 us (131 with full
// divisions and each product made twice).  Its gradient with dsum, 16,384 x
// 4096 (537 MB) 96 us, 5.6 TB/s, and 7.5 for the weight's partials: 118 without the
// next row's loads ahead, or with them and 130 registers instead of 128.  64 x 4096
// to 8 bits 4.4 us, 500 x 2560 fp32 gradient 6.7 + 4.1.  All by a trace of the
// kernels; in a loop the calls take 91 and 101 us, and 97 for 60,000 x 2048.
#include <type_traits>

#include "arith.hpp"
#include "lanes.hpp"
#include "launch.hpp"
#include "rows.hpp"
#include "step_launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kMaxBlocks = 1u << 21;    // of up to 1024 lanes: they are counted in 32 bits
constexpr uint32_t kPartials = 1024;         // workgroups of 4 waves that leave a row of partial sums

struct Norm {
  const void* x;
  size_t xstride;
  const void* residual;      // or the gradient that arrives at h
  size_t rstride;
  const void* weight;
  void* sum;
  size_t sstride;
  void* out;
  size_t ostride;
  float* scales;
  size_t cstride;
  const void* dout;
  size_t dstride;
  float* partials;           // NULL: no gradient of the weight
  size_t ntokens;
  uint32_t dim, group, groups;   // group: columns, the row's width or more for one
  uint32_t wbf16;
  float eps, width, per_width;   // the row's width and 1 / it
  float least;                   // squares below it are summed again, larger
};

template <uint32_t LPR>
constexpr uint32_t threads_of() {
  return LPR > kThreads ? LPR : kThreads;
}

// The N weights from column c on.
template <typename T>
__device__ __forceinline__ void load_weight(const Norm& n, uint32_t c, float* w) {
  constexpr int N = T::kVec;
  if (n.wbf16) {
    if constexpr (N == 4) {
      typedef uint32_t vec2_u __attribute__((ext_vector_type(2), aligned(2)));
      const vec2_u v = *reinterpret_cast<const vec2_u*>(elem<BF16>(n.weight, c));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[2 * i] = bits_f32(v[i] << 16);
        w[2 * i + 1] = bits_f32(v[i] & 0xFFFF0000u);
      }
    } else if constexpr (N == 8) {
      BF16::unpack(load_vec<BF16>(elem<BF16>(n.weight, c)), w);
    } else {
      w[0] = BF16::widen(*elem<BF16>(n.weight, c));
    }
  } else {
    if constexpr (N == 1) {
      w[0] = F32::widen(*elem<F32>(n.weight, c));
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) F32::unpack(load_vec<F32>(elem<F32>(n.weight, c + i)), w + i);
    }
  }
}

// The larger of two values that are not negative; a NaN is above all.
struct MaxBits {
  __device__ __forceinline__ float operator()(float a, float b) const { return bits_f32(max(f32_bits(a), f32_bits(b))); }
};

// The largest of `lanes` (4 to 64) neighbouring lanes' values, none negative.
__device__ __forceinline__ float max_lanes(float v, uint32_t lanes) {
  auto op = [](uint32_t a, uint32_t b) { return max(a, b); };
  uint32_t x = join_lanes<4>(f32_bits(v), op);
  if (lanes > 4) x = join_step<4>(x, op);
  if (lanes > 8) x = join_step<8>(x, op);
  if (lanes > 16) x = join_step<16>(x, op);
  if (lanes > 32) x = join_step<32>(x, op);
  return bits_f32(x);
}

// Two values joined over the LPR lanes of a row, in all of them.  lds: a
// workgroup's, another part for each call until a barrier.
template <uint32_t LPR, typename A, typename B>
__device__ __forceinline__ void join_row(float& a, float& b, float* lds) {
  a = join_lanes<(LPR < 64 ? LPR : 64)>(a, A{});
  b = join_lanes<(LPR < 64 ? LPR : 64)>(b, B{});
  if constexpr (LPR > 64) {      // the workgroup's one row
    static_assert(LPR == threads_of<LPR>(), "a row of several waves is a workgroup's");
    constexpr uint32_t W = LPR / 64;
    const uint32_t wave = threadIdx.x >> 6;
    if (lane_id() == 0) {
      lds[wave] = a;
      lds[W + wave] = b;
    }
    __syncthreads();
    a = lds[0];
    b = lds[W];
#pragma unroll
    for (uint32_t w = 1; w < W; ++w) {
      a = A{}(a, lds[w]);
      b = B{}(b, lds[W + w]);
    }
  }
}

// 1 / sqrt(x), also of subnormal x.
__device__ __forceinline__ float inverse_root(float x) {
  const bool small = x < 0x1p-100f;
  return __builtin_amdgcn_rsqf(small ? x * 0x1p64f : x) * (small ? 0x1p32f : 1.0f);
}
// Whether it holds for one of a wave's rows (a row of several waves: in all of them).
template <uint32_t LPR>
__device__ __forceinline__ bool any_row(bool b) {
  return LPR >= 64 ? b : (bool)__any(b);
}
// A row whose squares pass what fp32 holds, or fall below what it holds beside an
// eps as small, is summed once more, of values f times as large: below 2^-80 the
// squares that are lost count (32,768 of 2^-149), and 2^96 brings the smallest
// square up to 2^-106 and the sums not past 2^112.
// (x - x is 0 for what is finite, which takes no constant's register: past 96
// scalar ones a SIMD holds 7 of the kernel's waves and not 8, and 60,000 x 2048
// bf16 to 8 bits take 106 us and not 97.)
__device__ __forceinline__ bool finite(float x) { return x - x == 0.0f; }
__device__ __forceinline__ bool off_fp32(const Norm& n, float squares) { return !finite(squares) || squares < n.least; }
__device__ __forceinline__ float factor_of(bool off, float squares) {
  return !off ? 1.0f : squares > 1.0f ? 0x1p-80f : 0x1p96f;
}
// 1 / sqrt(mean of squares + eps) / f for the squares of f times the values: an
// infinity's is 0.
__device__ __forceinline__ float inverse(const Norm& n, float squares, float f) {
  const float mean = f == 1.0f || finite(squares) ? quotient(squares, n.width, n.per_width) : squares;
  return inverse_root(mean + n.eps * f * f);
}

// N e4m3 codes, nearest.
template <int N, bool NT>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* f, uint32_t skip) {
  if constexpr (N == 1) {
    *p = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[0], 0, false);
  } else {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], lo, true);
    }
    if (skip == 0) {
      if constexpr (N == 4) {
        typedef uint32_t word_u __attribute__((aligned(1)));
        if constexpr (NT)
          __builtin_nontemporal_store(w[0], reinterpret_cast<word_u*>(p));
        else
          *reinterpret_cast<word_u*>(p) = w[0];
      } else {
        typedef uint32_t vec2_u __attribute__((ext_vector_type(2), aligned(1)));
        if constexpr (NT)
          __builtin_nontemporal_store(vec2_u{w[0], w[1]}, reinterpret_cast<vec2_u*>(p));
        else
          *reinterpret_cast<vec2_u*>(p) = vec2_u{w[0], w[1]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((uint32_t)i >= skip) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  }
}

// By the steps of the first sum, so that a row beside one that needs this keeps
// its bits.
template <typename T, int U>
__device__ __forceinline__ float squares_of(const typename T::vec* v, const uint32_t* skip, float f) {
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float h[T::kVec];
    T::unpack(v[u], h);
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) {
      const float x = h[i] * f, s = __builtin_fmaf(x, x, sum);
      sum = (uint32_t)i >= skip[u] ? s : sum;
    }
  }
  return sum;
}

// Q8: rows of 8 bits.  LPR lanes have a row, U vectors each.
template <typename T, uint32_t LPR, int U, bool Q8, bool NT>
__global__ void __launch_bounds__(threads_of<LPR>()) norm_kernel(Norm n) {
  constexpr int N = T::kVec;
  constexpr uint32_t RPW = threads_of<LPR>() / LPR;
  __shared__ float lds[2][LPR > 64 ? 2 * LPR / 64 : 1];
  const uint32_t slot = threadIdx.x / LPR, lane = threadIdx.x % LPR;
  uint32_t turn = 0;
  for (size_t first = (size_t)blockIdx.x * RPW; first < n.ntokens; first += (size_t)gridDim.x * RPW) {
    const bool there = first + slot < n.ntokens;
    const size_t t = there ? first + slot : n.ntokens - 1;    // a spare slot computes the last row and writes nothing
    typename T::vec v[U], add[U];
    uint32_t at[U], skip[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = (u * LPR + lane) * N;
      at[u] = c < n.dim ? vec_at<T>(c, n.dim) : 0;
      skip[u] = c < n.dim ? c - at[u] : N;                    // a vector moved back counts its own elements only
      v[u] = zero_vec<T>();
      if (c < n.dim) v[u] = load_vec<T, NT>(elem<T>(n.x, t * n.xstride + at[u]));
    }
    if (n.residual) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        add[u] = zero_vec<T>();
        if (skip[u] < N) add[u] = load_vec<T, NT>(elem<T>(n.residual, t * n.rstride + at[u]));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float a[N], b[N];
        T::unpack(v[u], a);
        T::unpack(add[u], b);
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] += b[i];
        v[u] = T::pack(a);
      }
    }
    float squares = 0.0f, top = 0.0f;
    float peak[U], prod[Q8 ? U : 1][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float h[N];
      T::unpack(v[u], h);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float s = __builtin_fmaf(h[i], h[i], squares);
        squares = (uint32_t)i >= skip[u] ? s : squares;
      }
      peak[u] = 0.0f;
      if constexpr (Q8) {
        if (skip[u] < N) {
          float w[N];
          load_weight<T>(n, at[u], w);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            prod[u][i] = h[i] * w[i];
            if ((uint32_t)i >= skip[u]) peak[u] = MaxBits{}(fabsf(prod[u][i]), peak[u]);
          }
        }
        top = MaxBits{}(peak[u], top);
      }
    }
    join_row<LPR, SumOp, MaxBits>(squares, top, lds[turn]);
    turn ^= 1;
    float r = inverse(n, squares, 1.0f);
    float ks[2] = {1.0f, r * (1.0f / 448.0f)};      // a group's scale is its largest by these two
    if (const bool off = off_fp32(n, squares); __builtin_expect(any_row<LPR>(off), 0)) {
      const float f = factor_of(off, squares);
      float none = 0.0f;
      squares = squares_of<T, U>(v, skip, f);
      join_row<LPR, SumOp, SumOp>(squares, none, lds[turn]);
      turn ^= 1;
      r = f * inverse(n, squares, f);
      // of large rows r / 448 may be subnormal, and of one of zeroes without an eps r is infinite
      ks[0] = f < 1.0f ? 1.0f / 448.0f : 1.0f;
      ks[1] = squares == 0.0f ? 0.0f : f < 1.0f ? r : r * (1.0f / 448.0f);
    }
    if constexpr (Q8) {
      const uint32_t lanes = min(n.group / N, min(LPR, 64u));
#pragma unroll
      for (int u = 0; u < U; ++u) peak[u] = n.groups > 1 ? max_lanes(peak[u], lanes) : top;
    }
    if (!there) continue;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (skip[u] == N) continue;
      float h[N], w[N];
      if (n.sum) store_vec<T, NT>(elem<T>(n.sum, t * n.sstride + at[u]), v[u]);
      if constexpr (Q8) {
        // a group of tiny values is brought up first, so that 448 / a stays finite,
        // and one of the largest down, whose reciprocal would be subnormal
        float a = peak[u];
        if (__builtin_expect(__any((f32_bits(a) - f32_bits(0x1p-64f)) >> 30), 0)) {
          const float lift = a > 1.0f ? 0x1p-64f : 0x1p64f;
          a *= lift;
#pragma unroll
          for (int i = 0; i < N; ++i) prod[u][i] *= lift;
        }
        const float inv = a > 0.0f ? quotient(448.0f, a, reciprocal(a)) : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = prod[u][i] * inv;
        store_codes<N, NT>(static_cast<uint8_t*>(n.out) + t * n.ostride + at[u], h, skip[u]);
        const uint32_t c = at[u] + skip[u];
        if (c % n.group == 0)
          n.scales[t * n.cstride + c / n.group] = peak[u] * ks[0] * ks[1] + (peak[u] - peak[u]);      // no number for none
      } else {
        T::unpack(v[u], h);
        load_weight<T>(n, at[u], w);
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = h[i] * r * w[i];
        store_vec<T, NT>(elem<T>(n.out, t * n.ostride + at[u]), T::pack(h));
      }
    }
  }
}

// x is h here.  A row's loads are on their way while the row before it is
// summed and written, and the weights stay in registers where there is room.
template <typename T, uint32_t LPR, int U, bool NT>
__global__ void __launch_bounds__(threads_of<LPR>(), LPR >= 64 && LPR < 1024 && U * T::kVec == 16 ? 4 : 1) norm_grad_kernel(Norm n) {
  constexpr int N = T::kVec;
  constexpr uint32_t RPW = threads_of<LPR>() / LPR;
  constexpr bool kAhead = U * N <= 16 && LPR < 1024;
  __shared__ float lds[2][LPR > 64 ? 2 * LPR / 64 : 1];
  __shared__ float tile[RPW > 1 ? threads_of<LPR>() * U * N : 1];
  const uint32_t slot = threadIdx.x / LPR, lane = threadIdx.x % LPR;
  uint32_t turn = 0, at[U], skip[U];
  float dw[U][N], wk[kAhead ? U : 1][N];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t c = (u * LPR + lane) * N;
    at[u] = c < n.dim ? vec_at<T>(c, n.dim) : 0;
    skip[u] = c < n.dim ? c - at[u] : N;
#pragma unroll
    for (int i = 0; i < N; ++i) dw[u][i] = 0.0f;
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < N; ++i) wk[u][i] = 0.0f;
      if (skip[u] < N) load_weight<T>(n, at[u], wk[u]);
    }
  }
  struct Row {
    typename T::vec v[U], d[U], s[U];
  };
  auto load = [&](size_t first, Row& r) {
    const size_t t = first + slot < n.ntokens ? first + slot : n.ntokens - 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r.v[u] = r.d[u] = r.s[u] = zero_vec<T>();
      if (skip[u] < N) {
        r.v[u] = load_vec<T, NT>(elem<T>(n.x, t * n.xstride + at[u]));
        r.d[u] = load_vec<T, NT>(elem<T>(n.dout, t * n.dstride + at[u]));
        if (kAhead && n.residual) r.s[u] = load_vec<T, NT>(elem<T>(n.residual, t * n.rstride + at[u]));
      }
    }
  };
  Row row, next;
  const size_t step = (size_t)gridDim.x * RPW;
  load((size_t)blockIdx.x * RPW, row);
  for (size_t first = (size_t)blockIdx.x * RPW; first < n.ntokens; first += step) {
    const size_t t = first + slot;
    const bool there = t < n.ntokens, more = first + step < n.ntokens;
    if constexpr (kAhead)
      if (more) load(first + step, next);
    // Both sums, of h by f.  Written out twice, the first with f = 1: 16,384 x 4096
    // bf16 take 117 us and not 101 where the second reads the weights again, 128 where
    // a loop goes back with f (registers past 128 in either).
    float squares, dot, f = 1.0f;
    auto sums = [&] {
      squares = dot = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (skip[u] == N) continue;
        float h[N], dy[N], w[N];
        T::unpack(row.v[u], h);
        T::unpack(row.d[u], dy);
        if constexpr (!kAhead) load_weight<T>(n, at[u], w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if constexpr (kAhead) w[i] = wk[u][i];
          const float x = h[i] * f, a = __builtin_fmaf(x, x, squares), b = __builtin_fmaf(dy[i] * w[i], x, dot);
          squares = (uint32_t)i >= skip[u] ? a : squares;
          dot = (uint32_t)i >= skip[u] ? b : dot;
        }
      }
      join_row<LPR, SumOp, SumOp>(squares, dot, lds[turn]);
      turn ^= 1;
    };
    sums();
    if (const bool off = off_fp32(n, squares); any_row<LPR>(off)) {
      f = factor_of(off, squares);
      sums();
    }
    const float root = inverse(n, squares, f), r = f * root;
    dot = dot * n.per_width * root;
    if (there) {
      const float back = dot * r;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (skip[u] == N) continue;
        float h[N], dy[N], w[N], o[N];
        T::unpack(row.v[u], h);
        T::unpack(row.d[u], dy);
        if constexpr (!kAhead) {
          load_weight<T>(n, at[u], w);
          if (n.residual) row.s[u] = load_vec<T, NT>(elem<T>(n.residual, t * n.rstride + at[u]));
        }
        T::unpack(row.s[u], o);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if constexpr (kAhead) w[i] = wk[u][i];
          dw[u][i] = __builtin_fmaf(h[i] * r, dy[i], dw[u][i]);      // h r is near 1, however large the row
          o[i] = __builtin_fmaf(r, __builtin_fmaf(-back, h[i], dy[i] * w[i]), o[i]);
        }
        // a vector moved back stores its own elements only: the others' dsum
        // may be their dx already, another wave's
        if (skip[u] == 0) {
          store_vec<T, NT>(elem<T>(n.out, t * n.ostride + at[u]), T::pack(o));
        } else {
#pragma unroll
          for (int i = 1; i < N; ++i)
            if ((uint32_t)i >= skip[u]) *elem<T>(n.out, t * n.ostride + at[u] + i) = T::narrow(o[i]);
        }
      }
    }
    if (!more) break;
    if constexpr (kAhead)
      row = next;
    else
      load(first + step, row);
  }
  if (!n.partials) return;
  float* to = n.partials + (size_t)blockIdx.x * n.dim;
  if constexpr (RPW == 1) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (N > 1 && skip[u] == 0) {
#pragma unroll
        for (int i = 0; i + 4 <= N; i += 4) store_vec<F32>(elem<F32>(to, at[u] + i), F32::pack(dw[u] + i));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if ((uint32_t)i >= skip[u]) to[at[u] + i] = dw[u][i];
      }
    }
  } else {
    constexpr uint32_t wide = LPR * U * N;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((uint32_t)i >= skip[u]) tile[slot * wide + at[u] + i] = dw[u][i];
    }
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < n.dim; c += threads_of<LPR>()) {
      float sum = 0.0f;
#pragma unroll
      for (uint32_t k = 0; k < RPW; ++k) sum += tile[k * wide + c];
      to[c] = sum;
    }
  }
}

// The columns' partials added up: 16 columns a workgroup, by V (4, or 1 for
// fewer columns) in each of 64 (16) lanes that share a column's rows.
template <typename V, typename D>
__global__ void __launch_bounds__(kThreads) norm_dweight_kernel(const float* partials, uint32_t rows, uint32_t dim,
                                                                void* dweight, int accumulate) {
  constexpr uint32_t N = V::kVec, kLanes = 16 / N, kRows = kThreads / kLanes;
  __shared__ float tile[kWaves][16];
  const uint32_t c = blockIdx.x * 16 + threadIdx.x % kLanes * N, k = threadIdx.x / kLanes;
  const uint32_t at = c < dim ? vec_at<V>(c, dim) : 0;
  float sum[N];
#pragma unroll
  for (uint32_t i = 0; i < N; ++i) sum[i] = 0.0f;
  if (c < dim) {
#pragma unroll 8
    for (uint32_t r = k; r < rows; r += kRows) {
      float f[N];
      V::unpack(load_vec<V>(elem<V>(partials, (size_t)r * dim + at)), f);
#pragma unroll
      for (uint32_t i = 0; i < N; ++i) sum[i] += f[i];
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < N; ++i) {
#pragma unroll
    for (uint32_t m = kLanes; m < 64; m <<= 1) sum[i] += __shfl_xor(sum[i], (int)m);
    if (lane_id() < kLanes) tile[threadIdx.x >> 6][threadIdx.x % kLanes * N + i] = sum[i];
  }
  __syncthreads();
  if (threadIdx.x < kLanes && c < dim) {
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
      if (at + i < c) continue;        // of the vector before
      float total = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total += tile[w][threadIdx.x * N + i];
      typename D::raw* p = elem<D>(dweight, at + i);
      *p = D::narrow(accumulate ? D::widen(*p) + total : total);
    }
  }
}

// fn(T{}, lanes per row, vectors per lane) for a type and a width.
template <typename T, typename Fn>
hipError_t with_width(size_t dim, Fn fn) {
#define HC_ROW(L, U) fn(T{}, std::integral_constant<uint32_t, L>{}, std::integral_constant<int, U>{})
  if constexpr (T::kVec == 1) {
    return HC_ROW(8, 1);        // fewer columns than a vector has
  } else {
    const size_t vecs = (dim + T::kVec - 1) / T::kVec;
    if (vecs <= 8) return HC_ROW(8, 1);
    if (vecs <= 16) return HC_ROW(16, 1);
    if (vecs <= 32) return HC_ROW(32, 1);
    if (vecs <= 64) return HC_ROW(64, 1);
    if (vecs <= 128) return HC_ROW(64, 2);
    if (vecs <= 256) return HC_ROW(256, 1);
    if (vecs <= 512) return HC_ROW(256, 2);
    if (vecs <= 1024) return HC_ROW(512, 2);
    if (vecs <= 2048) return HC_ROW(1024, 2);
    if (vecs <= 4096) return HC_ROW(1024, 4);
    if constexpr (T::kVec == 4) return HC_ROW(1024, 8);
    return hipErrorInvalidValue;
  }
#undef HC_ROW
}
template <typename Fn>
hipError_t with_row(hc_dtype_t dtype, size_t dim, Fn fn) {
  if (dtype == HC_F32) return dim < F32::kVec ? with_width<F32S>(dim, fn) : with_width<F32>(dim, fn);
  return dim < BF16::kVec ? with_width<BF16S>(dim, fn) : with_width<BF16>(dim, fn);
}

Norm norm_of(const NormRows& a) {
  Norm n = {};
  n.x = a.x;
  n.xstride = a.xstride;
  n.residual = a.residual;
  n.rstride = a.rstride;
  n.weight = a.weight;
  n.wbf16 = a.wtype == HC_BF16;
  n.sum = a.sum;
  n.sstride = a.sstride;
  n.out = a.out;
  n.ostride = a.ostride;
  n.ntokens = a.ntokens;
  n.dim = (uint32_t)a.dim;
  n.eps = a.eps;
  n.width = (float)a.dim;
  n.per_width = 1.0f / n.width;
  n.least = n.eps < 0x1p-80f ? 0x1p-80f : 0.0f;
  return n;
}

}  // namespace

hipError_t launch_rms_norm(const NormRows& a, bool q8, uint32_t group, float* scales, size_t cstride,
                           hipStream_t stream) {
  Norm n = norm_of(a);
  n.scales = scales;
  n.cstride = cstride;
  n.groups = group ? (n.dim + group - 1) / group : 1;
  n.group = n.groups > 1 ? group : 1u << 30;
  const size_t es = a.dtype == HC_F32 ? 4 : 2, bytes = n.ntokens * n.dim * ((q8 ? 1 : es) + (n.sum ? es : 0));
  const bool nt = bytes >= kStreamStoreBytes;     // what is read is as much at least
  return with_row(a.dtype, a.dim, [&](auto type, auto lanes, auto vecs) {
    typedef decltype(type) T;
    constexpr uint32_t LPR = decltype(lanes)::value, TH = threads_of<LPR>();
    constexpr int U = decltype(vecs)::value;
    const uint64_t groups = (n.ntokens + TH / LPR - 1) / (TH / LPR);
    const uint32_t blocks = (uint32_t)(groups < kMaxBlocks ? groups : kMaxBlocks);
    auto launch = [&](auto kernel) {
      HC_ENQUEUE(kernel, blocks, TH, stream, n);
      return hipSuccess;
    };
    if (q8) return nt ? launch(norm_kernel<T, LPR, U, true, true>) : launch(norm_kernel<T, LPR, U, true, false>);
    return nt ? launch(norm_kernel<T, LPR, U, false, true>) : launch(norm_kernel<T, LPR, U, false, false>);
  });
}

size_t rms_norm_grad_ws_bytes(size_t ntokens, size_t dim) {
  return (ntokens < kPartials ? ntokens : kPartials) * dim * sizeof(float);
}

hipError_t launch_rms_norm_grad(const NormRows& a, const void* dout, size_t dstride, void* dweight, hc_dtype_t dwtype,
                                bool accumulate, void* ws, hipStream_t stream) {
  Norm n = norm_of(a);
  n.dout = dout;
  n.dstride = dstride;
  n.partials = dweight ? static_cast<float*>(ws) : nullptr;
  uint32_t rows = 0;
  if (n.ntokens) {
    const hipError_t e = with_row(a.dtype, a.dim, [&](auto type, auto lanes, auto vecs) {
      typedef decltype(type) T;
      constexpr uint32_t LPR = decltype(lanes)::value, TH = threads_of<LPR>();
      constexpr int U = decltype(vecs)::value;
      const uint64_t groups = (n.ntokens + TH / LPR - 1) / (TH / LPR);
      // As many waves, and fewer partials of wider rows.  Two rows a workgroup before
      // there are 8 waves a CU more: 500 x 2560 fp32 10.5 us by 256 workgroups, 11.8 by
      // 500; 1000 x 2048 bf16 9.8 and 12.4.  Not where a row waits for the one before
      // it: 200 x 12,000 bf16 14.2 by 128, 13.9 by 200.
      constexpr uint32_t most = kPartials * kThreads / TH, few = LPR < 1024 ? most / 2 : most;
      rows = (uint32_t)(groups <= few ? groups : groups >= 2 * most ? most : groups <= 2 * few ? few : (groups + 1) / 2);
      // rows read once, which the step before has mostly left in memory from here on
      if (n.ntokens * n.dim * sizeof(typename T::raw) >= kStreamStoreBytes)
        HC_ENQUEUE((norm_grad_kernel<T, LPR, U, true>), rows, TH, stream, n);
      else
        HC_ENQUEUE((norm_grad_kernel<T, LPR, U, false>), rows, TH, stream, n);
      return hipSuccess;
    });
    if (e != hipSuccess) return e;
  }
  if (!dweight) return hipSuccess;
  const uint32_t blocks = (n.dim + 15) / 16;
  auto launch = [&](auto kernel) {
    HC_ENQUEUE(kernel, blocks, kThreads, stream, n.partials, rows, n.dim, dweight, (int)accumulate);
    return hipSuccess;
  };
  if (n.dim < F32::kVec)
    return dwtype == HC_F32 ? launch(norm_dweight_kernel<F32S, F32>) : launch(norm_dweight_kernel<F32S, BF16>);
  return dwtype == HC_F32 ? launch(norm_dweight_kernel<F32, F32>) : launch(norm_dweight_kernel<F32, BF16>);
}

}  // namespace hc
