// grad_kernels.hip -- the norm of many gradient tensors taken as one vector,
// and clipping by it, for gfx950.
//
//   norm = sqrt(sum g^2)  or  max |g|;   out = round(min(1, max_norm / (norm + 1e-6)) * g)
//
// Both are streams over memory: the norm reads every element once, clipping
// reads it again and writes it.  The tensors are cut into chunks of 16 KB,
// numbered through all tensors, so that one launch covers a thousand small
// vectors and a large matrix evenly; a chunk's tensor is found by a search
// over the tensors' first chunks.  The table of tensors travels in the kernel's
// own arguments (up to kBatch tensors) or in the workspace, which a launch per
// kPacked tensors fills; no host memory has to outlive the call.
//
// Squares are summed in fp64: a product of two fp32 values is exact there and
// can neither overflow nor vanish, and the sum's rounding stays far below the
// result's; it costs nothing, since the pass waits for memory either way (1 GiB
// summed in 153 us with fp64, 151 with fp32).  Each workgroup leaves one
// partial; they are added in a fixed order, by the clipping launch's own
// workgroups up to 128 MB of gradients, by a launch between the two above it.
//
// Measured on 2^29 bf16 values in 450 tensors, outputs at odd elements: norm
// 162 us (6.6 TB/s; plain loads 172-210), clipping 350-360 us (6.0 TB/s;
// persistent workgroups with plain stores 430); 525 us a call.  2^25 values in
// 290 views of two buckets, mixed types: 14 + 26 us, 41 us a call.  A sum by whichever
// workgroup ends last, behind agent-scope atomics, took the norm pass from 19
// to 96 us.
#include "launch.hpp"
#include "rows.hpp"
#include "step_launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kChunkBytes = 16384;
constexpr uint32_t kVecs = kChunkBytes / 16 / kThreads;   // 16-byte vectors per lane and chunk
constexpr uint32_t kBatch = 128;        // tensors per kernel argument: 3.6 KB of the 4 KB
constexpr uint32_t kMaxGrid = 2048;     // 8 workgroups of 4 waves on each of 256 CUs
constexpr uint32_t kMostBlocks = 1u << 23;   // of a launch: its lanes are counted in 32 bits
constexpr uint32_t kStreamChunks = (uint32_t)(kStreamStoreBytes / kChunkBytes);
// The norm reads non-temporal, but for sizes whose clipping stores
// non-temporal: that leaves the caches to the gradients, which plain reads keep
// for it, until from here on they only push each other out.  Both passes on
// bf16 values, plain / non-temporal, us: 67 MB 40.7 / 38.9, 101 MB 57.1 / 55.5,
// 134 MB 65.7 / 70.0, 268 MB 126 / 134, 403 MB 193 / 198, 537 MB 265 / 263,
// 1.07 GB 549 / 531.  hc_grad_norm reads by the same rule, for the hc_clip_grads
// that follows it (134 MB 67 / 71, 268 MB 126 / 135, 403 MB 195 / 200, 500 MB 246 /
// 246 together); by itself it would be faster non-temporal (134 MB 27.7 / 25.5,
// 268 MB 48.6 / 44.3, 403 MB 71 / 64; the input just written 27 / 27, 58 / 49, 93 / 73).
constexpr uint32_t kStreamLoadChunks = (512u << 20) / kChunkBytes;
// Up to here the clipping launch has at most kMaxGrid workgroups, which add the
// partials up themselves; above it has one per chunk.
constexpr uint32_t kFuseChunks = (128u << 20) / kChunkBytes;
constexpr uint64_t kBf16Bit = 1ull << 63;

struct Entry {
  const void* src;
  void* dst;          // src where nothing is written
  uint64_t count;     // elements; kBf16Bit: bf16
};
struct Batch {
  Entry e[kBatch];
  uint32_t first[kBatch];   // the first chunk of each tensor
};

// A chunk of a tensor begins where its output is 128-byte aligned (the first
// begins up to a line before the tensor), so that a wave's stores fill whole
// lines however the output lies; loads may straddle lines, stores must not:
// with outputs at odd elements the clipping of 2^29 bf16 values took 385 us
// on chunks counted from the tensor's start and takes 350-360 on these.
__host__ __device__ __forceinline__ uint32_t lead_bytes(const void* p) { return (uint32_t)((uintptr_t)p & 127u); }
__host__ __device__ __forceinline__ uint64_t chunks_of(const Entry& e) {
  const uint64_t bytes = (e.count & ~kBf16Bit) * (e.count & kBf16Bit ? 2 : 4);
  const uint32_t a = lead_bytes(e.src), b = lead_bytes(e.dst);
  return (bytes + (a > b ? a : b) + kChunkBytes - 1) / kChunkBytes;
}

// The table in the workspace: entries, then first chunks.
struct TableView {
  const Entry* e;
  const uint32_t* first;
};

// Up to kPacked tensors as a table launch's arguments, 18 bytes each: 48-bit
// addresses, and the count and type in what is left over.
constexpr uint32_t kPacked = 224;
struct Packed {
  uint64_t src[kPacked], dst[kPacked];    // bits 48..63: the count's bits 0..15 and 16..31
  uint16_t rest[kPacked];                 // the count's bits 32..46; bit 15: bf16
};

// Writes a batch's entries and first chunks.
__global__ void __launch_bounds__(kThreads) table_kernel(Packed b, uint32_t n, uint32_t first_chunk, Entry* e,
                                                         uint32_t* first) {
  __shared__ uint32_t lds[kWaves];
  const uint32_t i = threadIdx.x;
  constexpr uint64_t kAddress = (1ull << 48) - 1;
  Entry x = {nullptr, nullptr, 0};
  if (i < n) {
    x.src = reinterpret_cast<const void*>(b.src[i] & kAddress);
    x.dst = reinterpret_cast<void*>(b.dst[i] & kAddress);
    x.count = (b.src[i] >> 48) | (b.dst[i] >> 48) << 16 | (uint64_t)(b.rest[i] & 0x7FFFu) << 32;
    if (b.rest[i] & 0x8000u) x.count |= kBf16Bit;
  }
  const uint32_t mine = i < n ? (uint32_t)chunks_of(x) : 0;
  uint32_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(sum, d);
    if (lane_id() >= (uint32_t)d) sum += y;
  }
  if (lane_id() == 63) lds[threadIdx.x >> 6] = sum;
  __syncthreads();
  uint32_t before = first_chunk;
  for (uint32_t w = 0; w < (threadIdx.x >> 6); ++w) before += lds[w];
  if (i < n) {
    e[i] = x;
    first[i] = before + sum - mine;
  }
}

// The tensor that holds chunk c, the last whose first chunk is not after it:
// a search over 64 places at a time, one per lane, so two loads in turn find
// it among 4096 tensors.  Every lane of the wave calls it.
__device__ __forceinline__ uint32_t find(const uint32_t* first, uint32_t n, uint32_t c) {
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

template <bool INF>
__device__ __forceinline__ double join(double a, double b) {
  if constexpr (INF) return (a > b || a != a) ? a : b;
  return a + b;
}

// All lanes' values joined; the result is valid in thread 0.
template <bool INF>
__device__ __forceinline__ double block_join(double v, double* lds) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = join<INF>(v, __shfl_xor(v, m));
  if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = join<INF>(v, lds[w]);
  return v;
}

template <typename T, bool INF>
__device__ __forceinline__ void add_vec(vec4 v, double* acc, uint32_t& big) {
  if constexpr (INF) {
    // magnitudes order as integers, infinities after numbers and NaN after both
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T::kVec == 4) {
        big = max(big, v[i] & 0x7FFFFFFFu);
      } else {
        big = max(big, max((v[i] << 16) & 0x7FFFFFFFu, v[i] & 0x7FFF0000u));
      }
    }
  } else {
    float f[T::kVec];
    T::unpack(v, f);
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) {
      const double d = (double)f[i];
      acc[i & 3] = __builtin_fma(d, d, acc[i & 3]);
    }
  }
}

// Where chunk c lies: its tensor, and its first byte there (negative where the
// chunk begins before the tensor).  A full chunk lies inside the tensor whole.
struct Place {
  const void* src;
  void* dst;
  int64_t at, bytes;
  bool bf16, full;
};

// OUT: counted from the output's line, else from the input's.
template <bool OUT>
__device__ __forceinline__ Place place_of(const Entry* e, const uint32_t* first, uint32_t n, uint32_t c) {
  const uint32_t t = find(first, n, c);
  const Entry x = e[t];
  Place p;
  p.src = x.src;
  p.dst = x.dst;
  p.bf16 = (x.count & kBf16Bit) != 0;
  p.bytes = (int64_t)((x.count & ~kBf16Bit) << (p.bf16 ? 1 : 2));
  p.at = (int64_t)(c - first[t]) * kChunkBytes - lead_bytes(OUT ? x.dst : x.src);
  p.full = p.at >= 0 && p.at + kChunkBytes <= p.bytes;
  return p;
}

template <bool NT>
__device__ __forceinline__ void load_full(const Place& p, vec4* v) {
  const char* q = static_cast<const char*>(p.src) + p.at + threadIdx.x * 16;
#pragma unroll
  for (uint32_t u = 0; u < kVecs; ++u) {
    const vec4_u* w = reinterpret_cast<const vec4_u*>(q + u * kThreads * 16);
    v[u] = NT ? __builtin_nontemporal_load(w) : *w;
  }
}

// A chunk that its tensor's ends cut: fn(p, first element) for its vectors of
// type V (T, or Single<T> for a tensor narrower than one), the last one moved
// back to end with the chunk where that has room for it; skip: how many of its
// elements the vector before it had already.
template <typename V, typename Fn>
__device__ __forceinline__ void each_vec(const Place& p, Fn fn) {
  constexpr int64_t kSize = sizeof(typename V::raw);
  const int64_t lo = p.at < 0 ? 0 : p.at / kSize;
  const int64_t end = p.at + kChunkBytes < p.bytes ? p.at + kChunkBytes : p.bytes, hi = end / kSize;
  for (int64_t i = lo + threadIdx.x * V::kVec; i < hi; i += kThreads * V::kVec) {
    const int64_t at = i + V::kVec <= hi ? i : hi - V::kVec;
    fn((size_t)at, (int)(i - at));
  }
}
// Whether the cut chunk has room for a vector of T.
template <typename T>
__device__ __forceinline__ bool wide(const Place& p) {
  const int64_t lo = p.at < 0 ? 0 : p.at, hi = p.at + kChunkBytes < p.bytes ? p.at + kChunkBytes : p.bytes;
  return hi - lo >= (int64_t)(T::kVec * sizeof(typename T::raw));
}

template <typename T, bool INF>
__device__ __forceinline__ void norm_cut(const Place& p, double* acc, uint32_t& big) {
  auto add = [&](float f) {
    if constexpr (INF) {
      big = max(big, f32_bits(f) & 0x7FFFFFFFu);
    } else {
      const double d = (double)f;
      acc[0] = __builtin_fma(d, d, acc[0]);
    }
  };
  if (wide<T>(p)) {
    each_vec<T>(p, [&](size_t at, int skip) {
      float f[T::kVec];
      T::unpack(load_vec<T>(elem<T>(p.src, at)), f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i)
        if (i >= skip) add(f[i]);
    });
  } else {
    each_vec<Single<T>>(p, [&](size_t at, int) { add(T::widen(*elem<T>(p.src, at))); });
  }
}

template <bool INF, bool NT>
__device__ void norm_body(const Entry* e, const uint32_t* first, uint32_t n, uint32_t chunks, double* partials) {
  __shared__ double lds[kWaves];
  double acc[4] = {0, 0, 0, 0};
  uint32_t big = 0;
  uint32_t c = blockIdx.x;
  Place p = place_of<false>(e, first, n, c);
  for (;;) {
    vec4 v[kVecs];
    if (p.full) load_full<NT>(p, v);
    // the next chunk is looked up while this one's data are on their way
    c += gridDim.x;
    const bool more = c >= gridDim.x && c < chunks;
    Place next = p;
    if (more) next = place_of<false>(e, first, n, c);
    __builtin_amdgcn_sched_barrier(0);
    if (p.full) {
      if (p.bf16) {
#pragma unroll
        for (uint32_t u = 0; u < kVecs; ++u) add_vec<BF16, INF>(v[u], acc, big);
      } else {
#pragma unroll
        for (uint32_t u = 0; u < kVecs; ++u) add_vec<F32, INF>(v[u], acc, big);
      }
    } else if (p.bf16) {
      norm_cut<BF16, INF>(p, acc, big);
    } else {
      norm_cut<F32, INF>(p, acc, big);
    }
    if (!more) break;
    p = next;
  }
  double v = INF ? (double)bits_f32(big) : (acc[0] + acc[1]) + (acc[2] + acc[3]);
  v = block_join<INF>(v, lds);
  if (threadIdx.x == 0) partials[blockIdx.x] = v;
}

// The norm from the workgroups' partials, the same bits in every workgroup.
template <bool INF>
__device__ __forceinline__ float norm_of(const double* partials, uint32_t n) {
  __shared__ double lds[kWaves];
  double v = 0.0;
  for (uint32_t i = threadIdx.x; i < n; i += kThreads) v = join<INF>(v, partials[i]);
  v = block_join<INF>(v, lds);
  return INF ? (float)v : (float)sqrt(v);
}

template <bool INF, bool NT>
__global__ void __launch_bounds__(kThreads) norm_args_kernel(Batch b, uint32_t n, uint32_t chunks, double* partials) {
  norm_body<INF, NT>(b.e, b.first, n, chunks, partials);
}
template <bool INF, bool NT>
__global__ void __launch_bounds__(kThreads) norm_table_kernel(TableView t, uint32_t n, uint32_t chunks,
                                                              double* partials) {
  norm_body<INF, NT>(t.e, t.first, n, chunks, partials);
}

template <bool INF>
__global__ void __launch_bounds__(kThreads) finish_kernel(const double* partials, uint32_t n, float* norm) {
  const float v = norm_of<INF>(partials, n);
  if (threadIdx.x == 0) *norm = v;
}

__device__ __forceinline__ float clip_coef(float norm, float max_norm) {
  const float c = max_norm / (norm + 1e-6f);
  return c > 1.0f ? 1.0f : c;   // NaN stays NaN
}

template <typename T, bool NT>
__device__ __forceinline__ void scale_full(const Place& p, const vec4* v, float coef) {
  char* q = static_cast<char*>(p.dst) + p.at + threadIdx.x * 16;
#pragma unroll
  for (uint32_t u = 0; u < kVecs; ++u) {
    float f[T::kVec];
    T::unpack(v[u], f);
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) f[i] *= coef;
    store_vec<T, NT>(reinterpret_cast<typename T::raw*>(q + u * kThreads * 16), T::pack(f));
  }
}
// In place a vector must not scale what another has scaled already, so the
// last one writes its own elements only.
template <typename T>
__device__ __forceinline__ void scale_cut(const Place& p, float coef) {
  if (wide<T>(p)) {
    each_vec<T>(p, [&](size_t at, int skip) {
      if (skip) {
#pragma unroll
        for (int i = 0; i < T::kVec; ++i)
          if (i >= skip) *elem<T>(p.dst, at + i) = T::narrow(T::widen(*elem<T>(p.src, at + i)) * coef);
        return;
      }
      float f[T::kVec];
      T::unpack(load_vec<T>(elem<T>(p.src, at)), f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) f[i] *= coef;
      store_vec<T>(elem<T>(p.dst, at), T::pack(f));
    });
  } else {
    each_vec<Single<T>>(
        p, [&](size_t at, int) { *elem<T>(p.dst, at) = T::narrow(T::widen(*elem<T>(p.src, at)) * coef); });
  }
}

template <bool INF, bool NT>
__device__ void clip_body(const Entry* e, const uint32_t* first, uint32_t n, uint32_t chunks, const double* partials,
                          uint32_t npartials, float* norm, float max_norm) {
  uint32_t c = blockIdx.x;
  Place p = place_of<true>(e, first, n, c);
  vec4 v[kVecs];
  if (p.full) load_full<false>(p, v);     // on its way while the norm is added up
  float total;
  if (partials) {
    total = norm_of<INF>(partials, npartials);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  } else {
    total = *norm;
  }
  const float coef = clip_coef(total, max_norm);
  for (;;) {
    if (coef != 1.0f || p.dst != p.src) {
      if (p.full) {
        if (p.bf16)
          scale_full<BF16, NT>(p, v, coef);
        else
          scale_full<F32, NT>(p, v, coef);
      } else if (p.bf16) {
        scale_cut<BF16>(p, coef);
      } else {
        scale_cut<F32>(p, coef);
      }
    }
    c += gridDim.x;
    if (c < gridDim.x || c >= chunks) break;
    p = place_of<true>(e, first, n, c);
    if (p.full) load_full<false>(p, v);
  }
}

template <bool INF, bool NT>
__global__ void __launch_bounds__(kThreads) clip_args_kernel(Batch b, uint32_t n, uint32_t chunks,
                                                             const double* partials, uint32_t npartials, float* norm,
                                                             float max_norm) {
  clip_body<INF, NT>(b.e, b.first, n, chunks, partials, npartials, norm, max_norm);
}
template <bool INF, bool NT>
__global__ void __launch_bounds__(kThreads) clip_table_kernel(TableView t, uint32_t n, uint32_t chunks,
                                                              const double* partials, uint32_t npartials, float* norm,
                                                              float max_norm) {
  clip_body<INF, NT>(t.e, t.first, n, chunks, partials, npartials, norm, max_norm);
}

// Workspace: kMaxGrid partials, then the table.
constexpr size_t kPartialBytes = kMaxGrid * sizeof(double);
size_t table_bytes(size_t n) { return (n * sizeof(Entry) + n * sizeof(uint32_t) + 15) & ~(size_t)15; }

// The spans of tensors and their chunks, ready to launch with.
struct Plan {
  Batch batch;            // the spans, where they fit the arguments
  bool by_args = true;
  TableView view = {nullptr, nullptr};
  uint32_t n = 0, chunks = 0, grid = 0;
};

Entry entry_of(const void* const* grads, void* const* outs, const size_t* counts, const hc_dtype_t* dtypes, size_t i) {
  return Entry{grads[i], outs ? outs[i] : const_cast<void*>(grads[i]),
               (uint64_t)counts[i] | (dtypes[i] == HC_BF16 ? kBf16Bit : 0)};
}

// Hands fn the spans to work on, as entries: tensors that follow one another
// in memory, inputs and outputs alike, are one, as a bucket's views are (fp32
// and bf16 ones in buckets of their own, in any order).  290 views of two
// buckets are 2 spans, with no table launches: 41 us for 2^25 values, 48 as 290 tensors.
template <typename Fn>
hipError_t each_span(const void* const* grads, void* const* outs, const size_t* counts, const hc_dtype_t* dtypes,
                     size_t ntensors, Fn fn) {
  Entry open[2] = {};       // by type; count 0: none
  for (size_t i = 0; i < ntensors; ++i) {
    if (counts[i] == 0) continue;
    const int bf = dtypes[i] == HC_BF16;
    Entry x = entry_of(grads, outs, counts, dtypes, i);
    Entry& o = open[bf];
    const size_t bytes = (size_t)(o.count & ~kBf16Bit) * (bf ? 2 : 4);
    if (o.count && x.src == static_cast<const char*>(o.src) + bytes && x.dst == static_cast<char*>(o.dst) + bytes) {
      o.count += counts[i];
      continue;
    }
    if (o.count)
      if (hipError_t e = fn(o); e != hipSuccess) return e;
    o = x;
  }
  for (const Entry& o : open)
    if (o.count)
      if (hipError_t e = fn(o); e != hipSuccess) return e;
  return hipSuccess;
}

hipError_t make_plan(const void* const* grads, void* const* outs, const size_t* counts, const hc_dtype_t* dtypes,
                     size_t ntensors, void* ws, hipStream_t stream, Plan* p) {
  uint64_t chunks = 0;
  hipError_t e = each_span(grads, outs, counts, dtypes, ntensors, [&](const Entry& x) {
    if (((uintptr_t)x.src | (uintptr_t)x.dst) >> 48 || (x.count & ~kBf16Bit) >> 47) return hipErrorInvalidValue;
    ++p->n;
    chunks += chunks_of(x);
    return chunks > 0xFFFFFFFFull - kMaxGrid ? hipErrorInvalidValue : hipSuccess;   // 64 TB of gradients
  });
  if (e != hipSuccess) return e;
  p->chunks = (uint32_t)chunks;
  p->grid = p->chunks < kMaxGrid ? p->chunks : kMaxGrid;
  p->by_args = p->n <= kBatch;
  Entry* table = reinterpret_cast<Entry*>(static_cast<char*>(ws) + kPartialBytes);
  uint32_t* firsts = reinterpret_cast<uint32_t*>(table + p->n);
  p->view = TableView{table, firsts};
  Packed pack;
  uint32_t k = 0, done = 0, first = 0, next = 0;
  return each_span(grads, outs, counts, dtypes, ntensors, [&](const Entry& x) {
    if (p->by_args) {
      p->batch.e[k] = x;
      p->batch.first[k++] = next;
      next += (uint32_t)chunks_of(x);
      return hipSuccess;
    }
    const uint64_t c = x.count & ~kBf16Bit;
    pack.src[k] = (uint64_t)(uintptr_t)x.src | c << 48;
    pack.dst[k] = (uint64_t)(uintptr_t)x.dst | (c >> 16) << 48;
    pack.rest[k++] = (uint16_t)(c >> 32 | (x.count & kBf16Bit ? 0x8000u : 0));
    next += (uint32_t)chunks_of(x);
    if (k == kPacked || done + k == p->n) {
      HC_ENQUEUE(table_kernel, 1, kThreads, stream, pack, k, first, table + done, firsts + done);
      done += k;
      first = next;
      k = 0;
    }
    return hipSuccess;
  });
}

// The clipping launch; partials NULL: the norm is in *norm already.
template <bool INF>
hipError_t run_clip(const Plan& p, float max_norm, float* norm, const double* partials, hipStream_t stream) {
  const uint32_t grid = partials ? p.grid : p.chunks < kMostBlocks ? p.chunks : kMostBlocks;
  const uint32_t np = partials ? p.grid : 0;
  const bool nt = p.chunks >= kStreamChunks;
  if (p.by_args) {
    if (nt)
      HC_ENQUEUE((clip_args_kernel<INF, true>), grid, kThreads, stream, p.batch, p.n, p.chunks, partials, np, norm,
                 max_norm);
    else
      HC_ENQUEUE((clip_args_kernel<INF, false>), grid, kThreads, stream, p.batch, p.n, p.chunks, partials, np, norm,
                 max_norm);
  } else {
    if (nt)
      HC_ENQUEUE((clip_table_kernel<INF, true>), grid, kThreads, stream, p.view, p.n, p.chunks, partials, np, norm,
                 max_norm);
    else
      HC_ENQUEUE((clip_table_kernel<INF, false>), grid, kThreads, stream, p.view, p.n, p.chunks, partials, np, norm,
                 max_norm);
  }
  return hipSuccess;
}

template <bool INF>
hipError_t run(const Plan& p, bool clip, float max_norm, float* norm, double* partials, hipStream_t stream) {
  const bool nt = p.chunks < kStreamChunks || p.chunks >= kStreamLoadChunks;
  if (p.grid && p.by_args) {
    if (nt)
      HC_ENQUEUE((norm_args_kernel<INF, true>), p.grid, kThreads, stream, p.batch, p.n, p.chunks, partials);
    else
      HC_ENQUEUE((norm_args_kernel<INF, false>), p.grid, kThreads, stream, p.batch, p.n, p.chunks, partials);
  } else if (p.grid) {
    if (nt)
      HC_ENQUEUE((norm_table_kernel<INF, true>), p.grid, kThreads, stream, p.view, p.n, p.chunks, partials);
    else
      HC_ENQUEUE((norm_table_kernel<INF, false>), p.grid, kThreads, stream, p.view, p.n, p.chunks, partials);
  }
  if (clip && p.grid && p.chunks <= kFuseChunks) return run_clip<INF>(p, max_norm, norm, partials, stream);
  HC_ENQUEUE(finish_kernel<INF>, 1, kThreads, stream, partials, p.grid, norm);
  return clip && p.grid ? run_clip<INF>(p, max_norm, norm, nullptr, stream) : hipSuccess;
}

}  // namespace

size_t grad_norm_ws_bytes(size_t ntensors) { return kPartialBytes + table_bytes(ntensors); }

hipError_t launch_grad_norm(const void* const* grads, void* const* outs, const size_t* counts,
                            const hc_dtype_t* dtypes, size_t ntensors, hc_norm_t kind, float max_norm, float* d_norm,
                            void* ws, hipStream_t stream) {
  Plan p;
  if (hipError_t e = make_plan(grads, outs, counts, dtypes, ntensors, ws, stream, &p); e != hipSuccess) return e;
  double* partials = static_cast<double*>(ws);
  return kind == HC_NORM_INF ? run<true>(p, outs != nullptr, max_norm, d_norm, partials, stream)
                             : run<false>(p, outs != nullptr, max_norm, d_norm, partials, stream);
}

hipError_t launch_grad_clip(const void* const* grads, void* const* outs, const size_t* counts,
                            const hc_dtype_t* dtypes, size_t ntensors, float max_norm, const float* d_norm, void* ws,
                            hipStream_t stream) {
  Plan p;
  if (hipError_t e = make_plan(grads, outs, counts, dtypes, ntensors, ws, stream, &p); e != hipSuccess) return e;
  if (!p.grid) return hipSuccess;
  return run_clip<false>(p, max_norm, const_cast<float*>(d_norm), nullptr, stream);   // only read, without partials
}

}  // namespace hc
