// expert_kernels.hip -- tokens sorted by expert and back with weights, and
// the gradient of the way back, for gfx950.
//
//   sort:      slots t * k + j laid out by expert, stable, aligned per expert
//   dispatch:  rows[row(t, j)] = x[t]
//   combine:   out[t] = round(sum_j w[t, j] * rows[row(t, j)])
//   gradient:  drows[row(t, j)] = round(w[t, j] * dout[t]),  dw[t, j] = <dout[t], rows[row(t, j)]>
//
// All but the sort are streams over rows, organised by token: a wave reads a
// token's slice once and writes its k copies, or reads its k rows and writes
// one sum, so the side that is k times larger moves exactly once and the
// other is not read k times over.  (By row instead, gathering each row's
// token: 298 against 232 us for 16,384 x 8 rows of 4096 bf16.)  Sums run over j
// in order within a lane: no atomics.  The token's row numbers are loaded once
// into the wave's lanes and read from there as scalars, so every row's address
// is scalar.
#include <type_traits>

#include "key_sort.hpp"
#include "launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kMaxBlocks = 1u << 22;

inline uint32_t blocks_for(uint64_t waves) {
  const uint64_t b = (waves + kWaves - 1) / kWaves;
  return (uint32_t)(b < kMaxBlocks ? b : kMaxBlocks);
}

// ---------------------------------------------------------------- sort

struct Sort {
  KeySource src;
  uint32_t n, tile, tiles, experts, bits, align, rows;
  uint32_t* hist;
  int32_t* row_of_slot;
  int32_t* slot_of_row;
  int32_t* offsets;
  int32_t* counts;
};

__global__ void __launch_bounds__(kSortThreads) expert_histogram_kernel(Sort s) {
  __shared__ uint32_t lds[kMaxRadix];
  const size_t lo = (size_t)blockIdx.x * s.tile;
  const size_t hi = lo + s.tile < s.n ? lo + s.tile : s.n;
  tile_histogram(lds, s.experts, lo, hi, [&](size_t i) { return load_key(s.src, i); },
                 s.hist + (size_t)blockIdx.x * s.experts);
}

// SELF: a short input, which every workgroup counts for itself (no histogram launch).
template <bool SELF>
__global__ void __launch_bounds__(kSortThreads) expert_scatter_kernel(Sort s) {
  __shared__ uint32_t counts[kSortWaves * kMaxRadix];
  __shared__ uint32_t scan[kSortWaves];
  const size_t lo = (size_t)blockIdx.x * s.tile;
  const size_t hi = lo + s.tile < s.n ? lo + s.tile : s.n;
  const uint32_t e = threadIdx.x;
  auto digit = [&](size_t i) { return load_key(s.src, i); };
  const Run run = load_run(lo, hi, s.tile, digit);
  uint32_t before, total, used;
  if constexpr (SELF)
    self_sums(counts, s.experts, s.n, lo, run, e, digit, &before, &total);
  else
    tile_sums(s.hist, s.experts, s.tiles, blockIdx.x, e, &before, &total);
  const uint32_t padded = (total + s.align - 1) / s.align * s.align;
  const uint32_t first = block_scan(padded, scan, &used);
  if (blockIdx.x == 0) {
    if (e < s.experts) {
      s.offsets[e] = (int32_t)first;
      s.counts[e] = (int32_t)total;
    }
    if (e == 0) s.offsets[s.experts] = (int32_t)used;
  }
  // rows without a slot: each expert's padding, spread over the tiles (by the
  // expert's lane, or by its wave where it may be long), and what lies behind
  // the last expert
  const bool mine = e < s.experts && e % gridDim.x == blockIdx.x;
  if (s.align <= 64) {
    if (mine)
      for (uint32_t r = first + total; r < first + padded; ++r) s.slot_of_row[r] = -1;
  } else {
    for (uint64_t todo = __ballot(mine); todo; todo &= todo - 1) {
      const uint32_t at = (uint32_t)__builtin_ctzll(todo);
      const uint32_t end = lane_read(first + padded, at);
      for (uint32_t r = lane_read(first + total, at) + lane_id(); r < end; r += 64) s.slot_of_row[r] = -1;
    }
  }
  for (size_t r = (size_t)used + blockIdx.x * kSortThreads + e; r < s.rows; r += (size_t)gridDim.x * kSortThreads)
    s.slot_of_row[r] = -1;
  place_items(counts, s.experts, s.bits, run, first + before, digit,
              [&](size_t i, uint32_t d, uint32_t place) {
                const bool there = d != kNoKey && place < s.rows;
                s.row_of_slot[i] = there ? (int32_t)place : -1;
                if (there) s.slot_of_row[place] = (int32_t)i;
              });
}

// ---------------------------------------------------------------- rows

struct Rows {
  const int32_t* row_of_slot;
  const int32_t* offsets;
  const int32_t* counts;
  const float* weights;
  size_t ntokens;
  uint32_t k, experts, dim, slices;
  uint32_t rows_room;       // a row number outside of it counts as none
  const void* x;            // by token (dispatch), or dout
  size_t xstride;
  const void* rows;         // by row (combine, gradient)
  size_t rstride;
  void* out;                // by token (combine) or by row (dispatch, gradient)
  size_t ostride;
  float* dweights;
  uint32_t pad_units;       // per expert
  uint64_t padding, units;  // the padding's units, then the tokens'
};

// A wave zeroes every pad_units-th group of kPadRows rows of an expert's
// padding, rows [offset + count, next offset).  These units come first in a
// launch: as its last waves, one per expert, they were its tail.
constexpr uint32_t kPadRows = 4, kMaxPadUnits = 64;
template <typename T, bool NT>
__device__ __forceinline__ void zero_padding(const Rows& r, uint64_t unit) {
  const uint32_t e = (uint32_t)(unit / r.pad_units);
  const uint32_t end = min((uint32_t)r.offsets[e + 1], r.rows_room);
  for (uint32_t g = (uint32_t)(r.offsets[e] + r.counts[e]) + (uint32_t)(unit % r.pad_units) * kPadRows; g < end;
       g += r.pad_units * kPadRows) {
    for (uint32_t row = g; row < end && row < g + kPadRows; ++row) {
      typename T::raw* p = elem<T>(r.out, (size_t)row * r.ostride);
      for (uint32_t c = lane_id() * T::kVec; c < r.dim; c += 64 * T::kVec)
        store_vec<T, NT>(p + vec_at<T>(c, r.dim), zero_vec<T>());
    }
  }
}

// A wave copies a slice of U * 64 vectors of one token to its k rows.
// Measured, 16,384 tokens x 8 of 128 experts x 4096 bf16, rows padded to 32:
// 240 us for 1.23 GB, 5.1 TB/s; a probe that does nothing else takes 225-232 with
// its input out of memory, and writing the rows alone takes 187.  U = 1 or 4:
// 251 and 250 where 2 took 247.
template <typename T, int U, bool NT>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(Rows r) {
  const uint32_t lane = lane_id();
  for (uint64_t u = (uint64_t)blockIdx.x * kWaves + wave_id(); u < r.units; u += (uint64_t)gridDim.x * kWaves) {
    if (u < r.padding) {
      zero_padding<T, NT>(r, u);
      continue;
    }
    const size_t t = (u - r.padding) / r.slices;
    const uint32_t c0 = (uint32_t)((u - r.padding) % r.slices) * (U * 64 * T::kVec) + lane * T::kVec;
    const int32_t row = lane < r.k ? r.row_of_slot[t * r.k + lane] : -1;
    uint64_t there = __ballot((uint32_t)row < r.rows_room);
    if (!there) continue;
    typename T::vec v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t c = c0 + i * 64 * T::kVec;
      if (c < r.dim) v[i] = load_vec<T>(elem<T>(r.x, t * r.xstride + vec_at<T>(c, r.dim)));
    }
    while (there) {
      const uint32_t j = (uint32_t)__builtin_ctzll(there);
      there &= there - 1;
      const size_t base = (size_t)lane_read((uint32_t)row, j) * r.ostride;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t c = c0 + i * 64 * T::kVec;
        if (c < r.dim) store_vec<T, NT>(elem<T>(r.out, base + vec_at<T>(c, r.dim)), v[i]);
      }
    }
  }
}

// A wave sums a slice of 64 vectors of one token's rows, four rows in flight.
// Measured: 5003 tokens x 2 slots x 1031 fp32 11.4 us (62 MB); 16,384 x 8 x 4096
// bf16 210 us (1.2 GB, 5.8 TB/s), eight rows in flight 204 there and 2-10% more
// than four on small inputs.
template <typename T, bool WEIGHTED, bool NTL, bool NT>
__global__ void __launch_bounds__(kThreads) combine_kernel(Rows r) {
  constexpr int N = T::kVec, J = 4;
  const uint32_t lane = lane_id();
  for (uint64_t u = (uint64_t)blockIdx.x * kWaves + wave_id(); u < r.units; u += (uint64_t)gridDim.x * kWaves) {
    const size_t t = u / r.slices;
    const uint32_t c = (uint32_t)(u % r.slices) * (64 * N) + lane * N;
    const int32_t row = lane < r.k ? r.row_of_slot[t * r.k + lane] : -1;
    const uint32_t w = WEIGHTED && lane < r.k ? f32_bits(r.weights[t * r.k + lane]) : f32_bits(1.0f);
    uint64_t there = __ballot((uint32_t)row < r.rows_room);
    const bool mine = c < r.dim;    // every lane stays, for the lane reads below
    const uint32_t at = vec_at<T>(c, r.dim);
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    while (there) {
      typename T::vec v[J];
      float g[J];
#pragma unroll
      for (int q = 0; q < J; ++q) {
        g[q] = 0.0f;
        v[q] = zero_vec<T>();
        if (!there) continue;
        const uint32_t j = (uint32_t)__builtin_ctzll(there);
        there &= there - 1;
        g[q] = bits_f32(lane_read(w, j));
        const size_t base = (size_t)lane_read((uint32_t)row, j) * r.rstride;
        if (mine) v[q] = load_vec<T, NTL>(elem<T>(r.rows, base + at));
      }
#pragma unroll
      for (int q = 0; q < J; ++q) {
        float f[N];
        T::unpack(v[q], f);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = __builtin_fmaf(g[q], f[i], acc[i]);
      }
    }
    if (mine) store_vec<T, NT>(elem<T>(r.out, t * r.ostride + at), T::pack(acc));
  }
}

// A workgroup of WPT waves takes a token, the waves sharing its slices; each row's
// dot product is summed over a lane's slices, then over lanes and waves in a
// fixed order.  J slots at a time: their rows' loads are in flight together
// with the token's.
// Measured, 16384 tokens x 8 slots x 4096 bf16 (2.28 GB): 426 us, 5.4 TB/s, as
// a large copy; one wave per token 467, J = 2 or 8 448 and 443, plain loads of
// the rows 447, plain stores 485.
template <typename T, int WPT, bool NTL, bool NT>
__global__ void __launch_bounds__(WPT * 64) combine_grad_kernel(Rows r) {
  constexpr int N = T::kVec, J = 4;
  __shared__ float part[WPT][J];
  const uint32_t lane = lane_id(), wave = wave_id();
  const uint64_t pad_blocks = (r.padding + WPT - 1) / WPT;
  for (uint64_t u = blockIdx.x; u < r.units; u += gridDim.x) {
    if (u < pad_blocks) {
      if (u * WPT + wave < r.padding) zero_padding<T, NT>(r, u * WPT + wave);
      continue;
    }
    const size_t t = u - pad_blocks;
    const int32_t row = lane < r.k ? r.row_of_slot[t * r.k + lane] : -1;
    const uint32_t w = lane < r.k ? f32_bits(r.weights[t * r.k + lane]) : 0;
    uint64_t there = __ballot((uint32_t)row < r.rows_room);
    float dw = 0.0f;        // lane j: slot j's
    while (there) {
      float dot[J], g[J];
      uint32_t slot[J];
      size_t rbase[J], obase[J];
      int live = 0;
#pragma unroll
      for (int q = 0; q < J; ++q) {
        dot[q] = 0.0f;
        slot[q] = 64;
        g[q] = 0.0f;
        rbase[q] = obase[q] = 0;
        if (!there) continue;
        slot[q] = (uint32_t)__builtin_ctzll(there);
        there &= there - 1;
        const size_t at = lane_read((uint32_t)row, slot[q]);
        rbase[q] = at * r.rstride;
        obase[q] = at * r.ostride;
        g[q] = bits_f32(lane_read(w, slot[q]));
        live = q + 1;
      }
      for (uint32_t c = threadIdx.x * N; c < r.dim; c += WPT * 64 * N) {
        typename T::vec v[J];
        const uint32_t at = vec_at<T>(c, r.dim), skip = c - at;
        const typename T::vec d = load_vec<T>(elem<T>(r.x, t * r.xstride + at));
#pragma unroll
        for (int q = 0; q < J; ++q) {
          v[q] = zero_vec<T>();
          if (q < live) v[q] = load_vec<T, NTL>(elem<T>(r.rows, rbase[q] + at));
        }
        float fd[N];
        T::unpack(d, fd);
#pragma unroll
        for (int q = 0; q < J; ++q) {
          if (q >= live) continue;
          float f[N], o[N];
          T::unpack(v[q], f);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            // a vector moved back counts its own elements only
            const float more = __builtin_fmaf(fd[i], f[i], dot[q]);
            dot[q] = (uint32_t)i >= skip ? more : dot[q];
            o[i] = g[q] * fd[i];
          }
          store_vec<T, NT>(elem<T>(r.out, obase[q] + at), T::pack(o));
        }
      }
#pragma unroll
      for (int q = 0; q < J; ++q) {
#pragma unroll
        for (int m = 32; m; m >>= 1) dot[q] += __shfl_xor(dot[q], m);
      }
      if constexpr (WPT > 1) {
        if (lane == 0) {
#pragma unroll
          for (int q = 0; q < J; ++q) part[wave][q] = dot[q];
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < J; ++q) {
          dot[q] = 0.0f;
#pragma unroll
          for (int w2 = 0; w2 < WPT; ++w2) dot[q] += part[w2][q];
        }
        __syncthreads();
      }
#pragma unroll
      for (int q = 0; q < J; ++q)
        if (lane == slot[q]) dw = dot[q];
    }
    if (wave == 0 && lane < r.k) r.dweights[t * r.k + lane] = dw;
  }
}

// fn(T{}) for the type, by single elements where a row is less than a vector.
template <typename Fn>
hipError_t with_type(hc_dtype_t dtype, size_t dim, Fn fn) {
  if (dtype == HC_F32) return dim < F32::kVec ? fn(F32S{}) : fn(F32{});
  return dim < BF16::kVec ? fn(BF16S{}) : fn(BF16{});
}

Rows rows_of(const hc_expert_plan_t& plan, size_t dim) {
  Rows r = {};
  r.row_of_slot = plan.row_of_slot;
  r.offsets = plan.expert_offsets;
  r.counts = plan.expert_counts;
  r.ntokens = plan.ntokens;
  r.k = (uint32_t)plan.k;
  r.experts = (uint32_t)plan.nexperts;
  r.dim = (uint32_t)dim;
  r.rows_room = (uint32_t)plan.rows;
  r.pad_units = ((uint32_t)plan.row_align - 1 + kPadRows - 1) / kPadRows;
  if (r.pad_units > kMaxPadUnits) r.pad_units = kMaxPadUnits;
  r.padding = (uint64_t)r.pad_units * r.experts;
  return r;
}

}  // namespace

size_t expert_sort_ws_bytes(size_t nslots, size_t nexperts) {
  // as if for kMaxTiles tiles: their number falls where a tile grows (64 at
  // 65,536 slots, 33 at 65,537), and a workspace has to do for fewer slots too
  return nslots <= kSelfCount ? 0 : (size_t)kMaxTiles * nexperts * sizeof(uint32_t);
}

hipError_t launch_expert_sort(const KeySource& src, const hc_expert_plan_t& plan, void* ws, hipStream_t stream) {
  Sort s = {};
  s.src = src;
  s.n = (uint32_t)(plan.ntokens * (size_t)plan.k);
  s.tile = sort_tile(s.n);
  s.tiles = sort_tiles(s.n);
  s.experts = (uint32_t)plan.nexperts;
  s.bits = 0;
  while ((s.experts - 1) >> s.bits) ++s.bits;
  s.align = (uint32_t)plan.row_align;
  s.rows = (uint32_t)plan.rows;
  s.hist = static_cast<uint32_t*>(ws);
  s.row_of_slot = plan.row_of_slot;
  s.slot_of_row = plan.slot_of_row;
  s.offsets = plan.expert_offsets;
  s.counts = plan.expert_counts;
  if (s.n <= kSelfCount) {
    HC_ENQUEUE(expert_scatter_kernel<true>, s.tiles ? s.tiles : 1, kSortThreads, stream, s);
    return hipSuccess;
  }
  HC_ENQUEUE(expert_histogram_kernel, s.tiles, kSortThreads, stream, s);
  HC_ENQUEUE(expert_scatter_kernel<false>, s.tiles, kSortThreads, stream, s);
  return hipSuccess;
}

hipError_t launch_expert_dispatch(const void* x, hc_dtype_t dtype, size_t dim, size_t xstride,
                                  const hc_expert_plan_t& plan, void* rows, size_t rstride, hipStream_t stream) {
  Rows r = rows_of(plan, dim);
  r.x = x;
  r.xstride = xstride;
  r.out = rows;
  r.ostride = rstride;
  return with_type(dtype, dim, [&](auto type) {
    typedef decltype(type) T;
    constexpr int U = 2;
    r.slices = (r.dim + U * 64 * T::kVec - 1) / (U * 64 * T::kVec);
    r.units = r.padding + (uint64_t)r.ntokens * r.slices;
    if (!r.units) return hipSuccess;
    const uint32_t blocks = blocks_for(r.units);
    // the rows in use number at most ntokens * k and the padding
    if (r.ntokens * r.k * r.dim * sizeof(typename T::raw) >= kStreamStoreBytes)
      HC_ENQUEUE((dispatch_kernel<T, U, true>), blocks, kThreads, stream, r);
    else
      HC_ENQUEUE((dispatch_kernel<T, U, false>), blocks, kThreads, stream, r);
    return hipSuccess;
  });
}

hipError_t launch_expert_combine(const void* rows, hc_dtype_t dtype, size_t dim, size_t rstride,
                                 const hc_expert_plan_t& plan, const float* weights, void* out, size_t ostride,
                                 hipStream_t stream) {
  Rows r = rows_of(plan, dim);
  r.rows = rows;
  r.rstride = rstride;
  r.weights = weights;
  r.out = out;
  r.ostride = ostride;
  return with_type(dtype, dim, [&](auto type) {
    typedef decltype(type) T;
    r.slices = (r.dim + 64 * T::kVec - 1) / (64 * T::kVec);
    r.units = (uint64_t)r.ntokens * r.slices;
    if (!r.units) return hipSuccess;
    auto launch = [&](auto kernel) {
      HC_ENQUEUE(kernel, blocks_for(r.units), kThreads, stream, r);
      return hipSuccess;
    };
    const size_t bytes = r.ntokens * r.dim * sizeof(typename T::raw);
    const bool nts = bytes >= kStreamStoreBytes, ntl = bytes * r.k >= kStreamLoadBytes;
    auto pick = [&](auto weighted) {
      constexpr bool W = decltype(weighted)::value;
      if (ntl) return nts ? launch(combine_kernel<T, W, true, true>) : launch(combine_kernel<T, W, true, false>);
      return nts ? launch(combine_kernel<T, W, false, true>) : launch(combine_kernel<T, W, false, false>);
    };
    return weights ? pick(std::true_type{}) : pick(std::false_type{});
  });
}

template <typename T, int WPT>
static hipError_t run_combine_grad(Rows r, hipStream_t stream) {
  r.units = (r.padding + WPT - 1) / WPT + r.ntokens;
  if (!r.units) return hipSuccess;
  const uint32_t blocks = (uint32_t)(r.units < kMaxBlocks ? r.units : kMaxBlocks);
  const size_t bytes = r.ntokens * r.k * r.dim * sizeof(typename T::raw);
  static_assert(kStreamLoadBytes >= kStreamStoreBytes, "streamed rows have streamed gradients");
  if (bytes >= kStreamLoadBytes)
    HC_ENQUEUE((combine_grad_kernel<T, WPT, true, true>), blocks, WPT * 64, stream, r);
  else if (bytes >= kStreamStoreBytes)
    HC_ENQUEUE((combine_grad_kernel<T, WPT, false, true>), blocks, WPT * 64, stream, r);
  else
    HC_ENQUEUE((combine_grad_kernel<T, WPT, false, false>), blocks, WPT * 64, stream, r);
  return hipSuccess;
}
template <typename T>
static hipError_t run_combine_grad(const Rows& r, hipStream_t stream) {
  // as many waves as a row has work for: 60000 tokens x 6 slots x 64 bf16 take
  // 55 us by one wave a token, 192 by four
  const uint32_t nvec = (r.dim + T::kVec - 1) / T::kVec;
  if (nvec <= 64) return run_combine_grad<T, 1>(r, stream);
  if (nvec <= 128) return run_combine_grad<T, 2>(r, stream);
  return run_combine_grad<T, 4>(r, stream);
}

hipError_t launch_expert_combine_grad(const void* dout, hc_dtype_t dtype, size_t dim, size_t dstride,
                                      const void* rows, size_t rstride, const hc_expert_plan_t& plan,
                                      const float* weights, void* drows, size_t drstride, float* dweights,
                                      hipStream_t stream) {
  Rows r = rows_of(plan, dim);
  r.x = dout;
  r.xstride = dstride;
  r.rows = rows;
  r.rstride = rstride;
  r.weights = weights;
  r.out = drows;
  r.ostride = drstride;
  r.dweights = dweights;
  return with_type(dtype, dim, [&](auto type) { return run_combine_grad<decltype(type)>(r, stream); });
}

}  // namespace hc
