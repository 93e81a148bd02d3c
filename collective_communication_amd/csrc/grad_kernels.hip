// grad_kernels.hip -- the norm of many gradient tensors taken as one vector,
// and clipping by it, for gfx950.
//
//   norm = sqrt(sum g^2)  or  max |g|;   out = round(min(1, max_norm / (norm + 1e-6)) * g)
//
// Both are streams over memory: the norm reads every element once, clipping
// reads it again and writes it.  The tensors are cut into chunks of 16 KB,
// numbered through all tensors, so that one launch covers a thousand small
// vectors and a large matrix evenly; a chunk's tensor is found by a binary
// search over the tensors' first chunks.  The table of tensors travels in the
// kernel's own arguments (up to kBatch tensors) or in the workspace, which a
// launch per kBatch tensors fills; no host memory has to outlive the call.
//
// Squares are summed in fp64: a product of two fp32 values is exact there and
// can neither overflow nor vanish, and the sum's rounding stays far below the
// result's.  Each workgroup leaves one partial; the partials are added in a
// fixed order, by the clipping kernel's workgroups themselves.
#include "launch.hpp"
#include "rows.hpp"
#include "step_launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kChunkBytes = 16384;
constexpr uint32_t kVecs = kChunkBytes / 16 / kThreads;   // 16-byte vectors per lane and chunk
constexpr uint32_t kBatch = 128;        // tensors per kernel argument: 3.6 KB of the 4 KB
constexpr uint32_t kMaxGrid = 2048;     // 8 workgroups of 4 waves on each of 256 CUs
constexpr uint64_t kBf16Bit = 1ull << 63;

struct Entry {
  const void* src;
  void* dst;
  uint64_t count;     // elements; kBf16Bit: bf16
};
struct Batch {
  Entry e[kBatch];
  uint32_t first[kBatch];   // the first chunk of each tensor
};

// The table in the workspace: entries, then first chunks.
struct TableView {
  const Entry* e;
  const uint32_t* first;
};

__global__ void __launch_bounds__(kBatch) table_kernel(Batch b, uint32_t n, Entry* e, uint32_t* first) {
  const uint32_t i = threadIdx.x;
  if (i < n) {
    e[i] = b.e[i];
    first[i] = b.first[i];
  }
}

// The tensor that holds chunk c: the last whose first chunk is not after it.
__device__ __forceinline__ uint32_t find(const uint32_t* first, uint32_t n, uint32_t c) {
  uint32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
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

template <typename T, bool INF>
__device__ __forceinline__ void norm_chunk(const void* src, uint64_t at, uint64_t count, double* acc, uint32_t& big) {
  constexpr uint32_t kElems = kChunkBytes / sizeof(typename T::raw);
  const uint64_t left = count - at;
  const typename T::raw* p = elem<T>(src, at);
  if (left >= kElems) {
    vec4 v[kVecs];
#pragma unroll
    for (uint32_t u = 0; u < kVecs; ++u)
      v[u] = *reinterpret_cast<const vec4_u*>(p + (size_t)(u * kThreads + threadIdx.x) * T::kVec);
#pragma unroll
    for (uint32_t u = 0; u < kVecs; ++u) add_vec<T, INF>(v[u], acc, big);
  } else {
    for (uint32_t i = threadIdx.x * T::kVec; i < left; i += kThreads * T::kVec)
      add_vec<T, INF>(load_vec<T>(p + i, (uint32_t)left - i), acc, big);
  }
}

template <bool INF>
__device__ void norm_body(const Entry* e, const uint32_t* first, uint32_t n, uint32_t chunks, double* partials) {
  __shared__ double lds[kWaves];
  double acc[4] = {0, 0, 0, 0};
  uint32_t big = 0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const uint32_t t = find(first, n, c);
    const Entry x = e[t];
    const uint64_t k = c - first[t];
    if (x.count & kBf16Bit)
      norm_chunk<BF16, INF>(x.src, k * (kChunkBytes / 2), x.count & ~kBf16Bit, acc, big);
    else
      norm_chunk<F32, INF>(x.src, k * (kChunkBytes / 4), x.count, acc, big);
  }
  double v = INF ? (double)bits_f32(big) : (acc[0] + acc[1]) + (acc[2] + acc[3]);
  v = block_join<INF>(v, lds);
  if (threadIdx.x == 0) partials[blockIdx.x] = v;
}

template <bool INF>
__global__ void __launch_bounds__(kThreads) norm_args_kernel(Batch b, uint32_t n, uint32_t chunks, double* partials) {
  norm_body<INF>(b.e, b.first, n, chunks, partials);
}
template <bool INF>
__global__ void __launch_bounds__(kThreads) norm_table_kernel(TableView t, uint32_t n, uint32_t chunks,
                                                              double* partials) {
  norm_body<INF>(t.e, t.first, n, chunks, partials);
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

template <bool INF>
__global__ void __launch_bounds__(kThreads) finish_kernel(const double* partials, uint32_t n, float* norm) {
  const float v = norm_of<INF>(partials, n);
  if (threadIdx.x == 0) *norm = v;
}

__device__ __forceinline__ float clip_coef(float norm, float max_norm) {
  const float c = max_norm / (norm + 1e-6f);
  return c > 1.0f ? 1.0f : c;   // NaN stays NaN
}

template <typename T>
__device__ __forceinline__ void clip_chunk(const Entry& x, uint64_t at, uint64_t count, float coef) {
  constexpr uint32_t kElems = kChunkBytes / sizeof(typename T::raw);
  const uint64_t left = count - at;
  const typename T::raw* p = elem<T>(x.src, at);
  typename T::raw* q = elem<T>(x.dst, at);
  if (left >= kElems) {
    vec4 v[kVecs];
#pragma unroll
    for (uint32_t u = 0; u < kVecs; ++u)
      v[u] = *reinterpret_cast<const vec4_u*>(p + (size_t)(u * kThreads + threadIdx.x) * T::kVec);
#pragma unroll
    for (uint32_t u = 0; u < kVecs; ++u) {
      float f[T::kVec];
      T::unpack(v[u], f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) f[i] *= coef;
      *reinterpret_cast<vec4_u*>(q + (size_t)(u * kThreads + threadIdx.x) * T::kVec) = T::pack(f);
    }
  } else {
    for (uint32_t i = threadIdx.x * T::kVec; i < left; i += kThreads * T::kVec) {
      float f[T::kVec];
      T::unpack(load_vec<T>(p + i, (uint32_t)left - i), f);
#pragma unroll
      for (int j = 0; j < T::kVec; ++j) f[j] *= coef;
      store_vec<T>(q + i, T::pack(f), (uint32_t)left - i);
    }
  }
}

// Chunks from the last one down: the norm pass read those last, so they are
// the ones the caches still hold.
template <bool INF>
__device__ void clip_body(const Entry* e, const uint32_t* first, uint32_t n, uint32_t chunks, const double* partials,
                          uint32_t npartials, float* norm, float max_norm) {
  float v;
  if (partials) {
    v = norm_of<INF>(partials, npartials);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  } else {
    v = *norm;
  }
  const float coef = clip_coef(v, max_norm);
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const uint32_t c = chunks - 1 - i;
    const uint32_t t = find(first, n, c);
    const Entry x = e[t];
    if (coef == 1.0f && x.dst == x.src) continue;
    const uint64_t k = c - first[t];
    if (x.count & kBf16Bit)
      clip_chunk<BF16>(x, k * (kChunkBytes / 2), x.count & ~kBf16Bit, coef);
    else
      clip_chunk<F32>(x, k * (kChunkBytes / 4), x.count, coef);
  }
}

template <bool INF>
__global__ void __launch_bounds__(kThreads) clip_args_kernel(Batch b, uint32_t n, uint32_t chunks,
                                                             const double* partials, uint32_t npartials, float* norm,
                                                             float max_norm) {
  clip_body<INF>(b.e, b.first, n, chunks, partials, npartials, norm, max_norm);
}
template <bool INF>
__global__ void __launch_bounds__(kThreads) clip_table_kernel(TableView t, uint32_t n, uint32_t chunks,
                                                              const double* partials, uint32_t npartials, float* norm,
                                                              float max_norm) {
  clip_body<INF>(t.e, t.first, n, chunks, partials, npartials, norm, max_norm);
}

// Workspace: kMaxGrid partials, then the table.
constexpr size_t kPartialBytes = kMaxGrid * sizeof(double);
size_t table_bytes(size_t n) { return (n * sizeof(Entry) + n * sizeof(uint32_t) + 15) & ~(size_t)15; }

// The non-empty tensors and their chunks, ready to launch with.
struct Plan {
  Batch batch;            // the tensors, where they fit the arguments
  bool by_args = true;
  TableView view = {nullptr, nullptr};
  uint32_t n = 0, chunks = 0, grid = 0;
};

hipError_t make_plan(const void* const* grads, void* const* outs, const size_t* counts, const hc_dtype_t* dtypes,
                     size_t ntensors, void* ws, hipStream_t stream, Plan* p) {
  size_t live = 0;
  uint64_t chunks = 0;
  for (size_t i = 0; i < ntensors; ++i) {
    const uint64_t elems = kChunkBytes / (dtypes[i] == HC_BF16 ? 2 : 4);
    live += counts[i] != 0;
    chunks += (counts[i] + elems - 1) / elems;
    if (chunks > 0xFFFFFFFFull - kMaxGrid) return hipErrorInvalidValue;   // 64 TB of gradients
  }
  p->by_args = live <= kBatch;
  Entry* table = reinterpret_cast<Entry*>(static_cast<char*>(ws) + kPartialBytes);
  uint32_t* firsts = reinterpret_cast<uint32_t*>(table + live);
  uint32_t k = 0, done = 0;
  chunks = 0;
  for (size_t i = 0; i < ntensors; ++i) {
    if (counts[i] == 0) continue;
    const bool bf = dtypes[i] == HC_BF16;
    p->batch.e[k] = Entry{grads[i], outs ? outs[i] : nullptr, (uint64_t)counts[i] | (bf ? kBf16Bit : 0)};
    p->batch.first[k] = (uint32_t)chunks;
    const uint64_t elems = kChunkBytes / (bf ? 2 : 4);
    chunks += (counts[i] + elems - 1) / elems;
    ++k;
    ++p->n;
    if (!p->by_args && (k == kBatch || p->n == live)) {
      table_kernel<<<1, kBatch, 0, stream>>>(p->batch, k, table + done, firsts + done);
      if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
      done += k;
      k = 0;
    }
  }
  p->view = TableView{table, firsts};
  p->chunks = (uint32_t)chunks;
  p->grid = p->chunks < kMaxGrid ? p->chunks : kMaxGrid;
  return hipSuccess;
}

template <bool INF>
hipError_t run(const Plan& p, bool clip, float max_norm, float* norm, double* partials, hipStream_t stream) {
  if (p.grid) {
    if (p.by_args)
      norm_args_kernel<INF><<<p.grid, kThreads, 0, stream>>>(p.batch, p.n, p.chunks, partials);
    else
      norm_table_kernel<INF><<<p.grid, kThreads, 0, stream>>>(p.view, p.n, p.chunks, partials);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!clip || !p.grid)
    finish_kernel<INF><<<1, kThreads, 0, stream>>>(partials, p.grid, norm);
  else if (p.by_args)
    clip_args_kernel<INF><<<p.grid, kThreads, 0, stream>>>(p.batch, p.n, p.chunks, partials, p.grid, norm, max_norm);
  else
    clip_table_kernel<INF><<<p.grid, kThreads, 0, stream>>>(p.view, p.n, p.chunks, partials, p.grid, norm, max_norm);
  return hipGetLastError();
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
  float* norm = const_cast<float*>(d_norm);   // read only, without partials
  if (p.by_args)
    clip_args_kernel<false><<<p.grid, kThreads, 0, stream>>>(p.batch, p.n, p.chunks, nullptr, 0, norm, max_norm);
  else
    clip_table_kernel<false><<<p.grid, kThreads, 0, stream>>>(p.view, p.n, p.chunks, nullptr, 0, norm, max_norm);
  return hipGetLastError();
}

}  // namespace hc
